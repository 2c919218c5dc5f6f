"""Cases of the operators around the recurrence that are large enough for what
the launchers do with real sizes: long tiles, many slots, several sequences or
groups of heads a lane.  Each names what it is there for; test_layer_plans.py
checks on the CPU that it gets it, test_gpu_layer_sizes.py the results."""

LENGTHS = [0, 5, 700, 1, 64, 383, 0, 937]  # 2090 tokens: sequences end inside every tile length

# forward and backward tile
CONV = {
    "bf16": dict(D=8196, W=4, dtype="bf16", lengths=LENGTHS, act="silu", tiles=(16, 32)),
    "f32": dict(D=16390, W=3, dtype="f32", lengths=LENGTHS, act="silu", tiles=(16, 64)),
    "rows": dict(D=16384, W=2, dtype="bf16", B=3, T=701, act="none", tiles=(16, 64)),
}

# slots forward and backward, and whether sequences pass from one to the next
SCAN = {
    "many-slots": dict(B=1, T=0, D=80, N=16, dtype="f32", lengths=[3000, 17, 0, 1303, 4000], slots=(130, 130),
                       carry=True),
    "many-slots-rows": dict(B=4, T=544, D=20, N=48, dtype="bf16", slots=(34, 34), carry=True),
    "32-slots": dict(B=1, T=2048, D=144, N=12, G=2, dtype="bf16", slots=(32, 32), carry=True),
    "rows-alone": dict(B=24, T=70, D=1024, N=4, dtype="bf16", slots=(24, 14), carry=False),
}

# sequences a lane
STEP = {
    "vectors": dict(S=50, D=4096, N=16, G=1, dtype="bf16", seqs=3),
    "single-states": dict(S=49, D=4100, N=15, G=2, dtype="f32", seqs=3),
    "widest": dict(S=13, D=3840, N=64, G=2, dtype="bf16", seqs=3),
}

# groups of heads a wave takes of a token, and waves a token (forward; a power of two backward)
NORM = {
    "quads": dict(rows=(2, 2050), Hq=19, Hk=3, d=128, rot=64, dtype="bf16", steps=6, waves=1),
    "single-pairs": dict(rows=(1, 4100), Hq=9, Hk=3, d=34, rot=34, dtype="f32", steps=7, waves=1),
    "wide-head": dict(rows=(1, 4100), Hq=2, Hk=1, d=258, rot=0, dtype="bf16", steps=3, waves=1),
    "many-groups": dict(rows=(2100,), Hq=17, Hk=3, d=258, rot=66, dtype="f32", steps=16, waves=2),
}
