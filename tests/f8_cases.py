"""Sizes (M, N, K) of the FP8 products with block scales and the form that bf16 and fp32 output take on 256 CUs."""

FORMS = {
    "few": [(1, 16, 128), (1, 1, 1), (3, 40, 200), (16, 256, 512), (17, 33, 640), (33, 70, 1100), (64, 96, 513),
            (50, 1000, 384), (200, 100, 300), (1, 700, 5000), (513, 520, 260), (40, 8300, 700)],
    "128": [(1500, 1500, 200), (1153, 1985, 1300), (2000, 1111, 520), (4360, 4104, 300)],
    # one tile a workgroup, and several; K of odd and even numbers of 512
    "persistent": [(4000, 4000, 520), (3900, 4088, 1024), (8100, 4096, 300), (8000, 4096, 700)],
    # odd N, and (fp32 output) the sizes above
    "256": [(4000, 4091, 600)],
}
SHAPES = [s for v in FORMS.values() for s in v]
