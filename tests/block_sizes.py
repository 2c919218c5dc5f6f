"""Cases of linear attention whose tokens are cut into many slots, and the
slots that a device of 256 compute units gets of them."""

LINEAR = {
    # shorter slots than the states are worth, so that every unit has one
    "one-for-each-unit": dict(B=1, T=4500, Hq=1, H=1, dk=24, dv=16, dtype="bf16", slots=(64, 71)),
    # as many tokens as the states are worth
    "least-tokens": dict(B=1, T=2500, Hq=2, H=8, dk=16, dv=16, dtype="bf16", slots=(128, 20)),
    "least-tokens-f32": dict(B=2, T=1250, Hq=8, H=8, dk=8, dv=20, dtype="f32", slots=(128, 20)),
    # as many as every unit holds: three of 64 columns
    "three-for-each-unit": dict(B=1, T=8300, Hq=3, H=6, dk=16, dv=12, dtype="bf16", slots=(128, 65)),
    "three-packed": dict(B=1, T=0, Hq=2, H=6, dk=12, dv=16, dtype="bf16", lengths=[3000, 1, 0, 5400, 63, 64, 65],
                         slots=(128, 68)),
    "wide-slots": dict(B=1, T=600, Hq=2, H=12, dk=100, dv=72, dtype="bf16", slots=(64, 10)),
}


def tokens(c):
    return sum(c["lengths"]) if "lengths" in c else c["B"] * c["T"]


def case(name):
    return {k: v for k, v in LINEAR[name].items() if k != "slots"}
