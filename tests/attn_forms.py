"""Sizes of calls for every form of launch that the attention over the 4-bit cache has
(csrc/attn_plan.h), each with its planner's answer: test_attn_plan_host.py holds the
planner to it, test_gpu_attn_kv4.py runs them."""

# kv_len, new tokens and heads of a call; `plan`: tiles to a prompt's workgroup, eight waves, split
FORMS = {
    "eight waves": dict(kv_len=[300, 77, 170], new=[1, 5, 3], heads=4, kv_heads=2, max_kv=640,
                        window=100, sinks=5, dims=(64, 128), plan=(0, 1, False)),
    "split": dict(kv_len=[9000, 5000], new=[1, 2], heads=4, kv_heads=1, max_kv=9000,
                  window=1900, sinks=5, dims=(64, 128, 256), plan=(0, 0, True)),
    "four waves": dict(kv_len=[70] * 129 + [200] * 15, new=[1] * 129 + [3] * 15, heads=6, kv_heads=2,
                       max_kv=256, window=66, sinks=2, dims=(64, 128, 256), plan=(0, 0, False)),
    "two tiles": dict(kv_len=[2500, 140], new=[300, 60], heads=124, kv_heads=2, max_kv=2560,
                      window=90, sinks=3, dims=(64, 128), plan=(2, 0, False)),
    "one tile": dict(kv_len=[2500, 140], new=[200, 30], heads=64, kv_heads=2, max_kv=2560,
                     window=1990, sinks=3, dims=(64, 128), plan=(1, 0, False)),
}


def sizes(f, dim, window):
    """The arguments of attn4_plan but for the type."""
    return (len(f["kv_len"]), sum(f["new"]), f["heads"], f["kv_heads"], dim, f["max_kv"],
            f["window"] if window else 0, f["sinks"] if window else 0)
