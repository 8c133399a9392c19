"""Calls that reach the kernel variants which small or ordinary calls do not: three and four
slots to a wave, three in the layout of pairs, 16-byte pieces of every row type, and partners of
the half-split rotation 1 and 32 lanes apart."""

# row type, T, heads_q, heads_k, head_dim, rot, interleaved, gamma stride, row padding (the
# cases of test_rope_gpu.py); then the layout and slots to a wave that the planner takes
ROPE = [
    (("bf16", 1100, 32, 32, 128, 128, False, 0, 0), ("whole", 4)),
    (("bf16", 2500, 10, 2, 128, 128, False, 0, 0), ("whole", 3)),
    (("bf16", 1100, 28, 28, 128, 64, True, 0, 0), ("whole", 4)),        # the last wave of a side: three slots
    (("bf16", 2500, 10, 2, 128, 128, True, 136, 8), ("whole", 3)),      # a gamma for each head
    (("f32", 1100, 16, 16, 128, 128, False, 0, 0), ("whole", 4)),
    (("f32", 2500, 5, 1, 128, 64, False, None, 0), ("whole", 3)),
    (("fp8", 1100, 32, 32, 128, 128, False, 0, 0), ("whole", 4)),
    (("fp8", 2500, 20, 4, 128, 128, True, 0, 0), ("whole", 3)),
    (("bf16", 3000, 10, 2, 80, 80, False, 0, 0), ("pairs", 3)),
    (("bf16", 3000, 10, 2, 96, 96, True, None, 0), ("pairs", 3)),
    (("bf16", 3000, 9, 3, 96, 32, False, 0, 0), ("pairs", 3)),
    (("f32", 3000, 5, 1, 80, 80, False, 0, 0), ("pairs", 3)),
    (("f32", 3000, 5, 1, 96, 96, False, 0, 0), ("pairs", 3)),
    (("fp8", 3000, 20, 4, 96, 96, False, 0, 0), ("pairs", 3)),
    (("fp8", 70, 3, 2, 96, 96, False, 0, 0), ("pairs", 1)),
    (("f32", 70, 3, 2, 96, 96, True, 0, 0), ("pairs", 1)),
    (("f32", 70, 3, 2, 256, 256, False, 0, 0), ("whole", 1)),           # partners 32 lanes apart
    (("bf16", 70, 3, 2, 512, 512, False, 0, 0), ("whole", 1)),
    (("bf16", 70, 3, 2, 128, 16, False, 0, 0), ("whole", 1)),           # 1 lane
    (("f32", 70, 3, 2, 64, 8, False, 0, 0), ("whole", 1)),
    (("f32", 70, 3, 2, 64, 16, False, 0, 0), ("whole", 1)),             # 2 lanes
]

# keyword arguments of test_paged_append_gpu.Case
APPEND = [
    (dict(dtype="bf16", T=1000, nq=12, nk=12, d=128, rot=128, inter=False), ("whole", 3)),
    (dict(dtype="bf16", T=1000, nq=11, nk=11, d=128, rot=64, inter=True, stride=128), ("whole", 3)),
    (dict(dtype="bf16", T=700, nq=16, nk=16, d=128, rot=128, inter=False, ps=64), ("whole", 4)),
    (dict(dtype="bf16", T=450, nq=28, nk=28, d=128, rot=128, inter=False, norm=False), ("whole", 4)),
    (dict(dtype="bf16", T=450, nq=28, nk=28, d=128, rot=128, inter=False), ("whole", 4)),
    (dict(dtype="f32", T=700, nq=8, nk=8, d=128, rot=128, inter=False), ("whole", 4)),
    (dict(dtype="bf16", T=1400, nq=12, nk=6, d=96, rot=96, inter=False), ("pairs", 3)),
    (dict(dtype="f32", T=1400, nq=8, nk=4, d=96, rot=96, inter=True), ("pairs", 3)),
    (dict(dtype="f32", T=50, nq=3, nk=2, d=256, rot=256, inter=False), ("whole", 1)),
    (dict(dtype="bf16", T=50, nq=3, nk=2, d=512, rot=512, inter=False), ("whole", 1)),
    (dict(dtype="bf16", T=50, nq=3, nk=2, d=128, rot=16, inter=False), ("whole", 1)),
    (dict(dtype="f32", T=50, nq=3, nk=2, d=32, rot=8, inter=False), ("whole", 1)),
]
