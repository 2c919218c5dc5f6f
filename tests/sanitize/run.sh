#!/bin/bash
# AddressSanitizer + UndefinedBehaviorSanitizer over the host-only code, on
# the CPU (no GPU): the C front ends kda_api.cpp and kda_layer_api.cpp (kernel
# launchers replaced by host_stubs.cpp and layer_stubs.cpp) and both oracle sources, built with g++/gcc, then the ABI
# tests and the oracle pins run against those builds.
#   bash tests/sanitize/run.sh [build-dir]
set -euo pipefail
R=$(cd "$(dirname "$0")/../.." && pwd)
O=${1:-/tmp/kda_sanitize}
mkdir -p "$O"
SAN="-fsanitize=address,undefined -fno-sanitize-recover=undefined -fno-omit-frame-pointer -g -O1"
g++ $SAN -std=c++17 -fPIC -shared -Wall -I"$R/include" -I"$R/gated_delta_rule_105_amd/csrc" -o "$O/libkda.so" "$R/gated_delta_rule_105_amd/csrc/kda_api.cpp" "$R/gated_delta_rule_105_amd/csrc/kda_layer_api.cpp" "$R/tests/sanitize/host_stubs.cpp" "$R/tests/sanitize/layer_stubs.cpp"
gcc $SAN -std=c99 -fPIC -shared -fopenmp -Wall -o "$O/libkda_oracle.so" "$R/oracle/kda_oracle.c" "$R/oracle/kda_oracle_bwd.c" -lm
export LD_PRELOAD="$(gcc -print-file-name=libasan.so) $(gcc -print-file-name=libubsan.so)"
export ASAN_OPTIONS=detect_leaks=0:abort_on_error=1
export UBSAN_OPTIONS=print_stacktrace=1:halt_on_error=1
export KDA_LIBRARY="$O/libkda.so" KDA_ORACLE_LIBRARY="$O/libkda_oracle.so"
cd "$R"
python -m pytest tests/test_abi.py tests/test_layer_abi.py tests/test_layer_abi_limits.py tests/test_oracle_pins.py tests/test_oracle_bwd_pins.py -q -s -m "not gpu" -p no:cacheprovider
