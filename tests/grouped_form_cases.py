"""Sizes that reach the forms of the grouped calls.  The host tests hold each of them against the library's own rules for
256 compute units, so that a rule that changes cannot move a case off its form unseen; the GPU tests run them."""

CUS = 256
RAGGED16 = [700, 0, 256, 1, 513, 900, 31, 300] * 2
# 70 groups, some empty, the second block of 64 with empty and full ones
RAGGED70 = [(i * 97) % 641 if i % 6 else 0 for i in range(70)]
# 300 groups: five blocks of 64
RAGGED300 = [(i * 89) % 541 if i % 7 else 0 for i in range(300)]

# (sizes of the groups, rows behind the last group, N, K, bias, {bf16 form, by the row stride's kind}, fp32 form)
PRODUCTS = {
    "16 groups": (RAGGED16, 300, 2720, 136, False, "persistent", "256"),
    "16 groups, bias": (RAGGED16, 300, 2720, 264, True, "persistent", "256"),
    "70 groups": (RAGGED70, 0, 320, 40, False, "persistent", "256"),
    "70 groups, bias, rows in no group": (RAGGED70, 700, 328, 520, True, "persistent", "256"),
    "70 groups, odd columns": (RAGGED70, 260, 323, 136, False, "persistent", "256"),
    "300 groups, bias": (RAGGED300, 1, 136, 72, True, "persistent", "256"),
    # a bias whose rows start off the 16-byte boundaries
    "16 groups, odd columns, bias": (RAGGED16, 5, 2723, 72, True, "256", "256"),
    # more groups than the persistent form's table holds
    "520 groups, bias": ([(i * 7) % 23 for i in range(519)] + [900], 95000, 136, 40, True, "256", "256"),
    "70 groups, few columns": (RAGGED70, 0, 72, 136, True, "128", "128"),
}

# (sizes, N, K, form of bf16)
WGRADS = {
    "520 groups": ([(i * 7) % 23 for i in range(519)] + [900], 40, 72, "256"),
    "300 groups": ([(i * 13) % 41 if i % 3 else 0 for i in range(300)], 136, 200, "persistent"),
}

BOTH = ["rne", "sr", "sr apart", "2d", "rht", "rht sr"]
ROWS = [0, 37, 700, 1, 64, 1500, 130, 800]
# (sizes, N, rows of x when gathered, both directions, options, form)
QUANTIZERS = {"tiles, %s, %d" % (o, n): (ROWS, n, 2000, True, o, "tiles")
              for n in (2600, 2608, 2595) for o in BOTH}
QUANTIZERS.update({"narrow, %s" % o: (ROWS[:5], 200, 300, True, o, "narrow") for o in BOTH[:4]})
for _name, _sizes in {"one row": [1], "few": [0, 1, 0, 33, 128, 0, 129, 5, 0], "block edges": [31, 32, 33, 127, 128, 129],
                      "70 groups": [(i * 7) % 23 for i in range(70)], "many": ROWS}.items():
    QUANTIZERS.update({"row-wise, %s, %s, %d" % (_name, o, n): (_sizes, n, 100, False, o, "tiles")
                       for n in (8, 136, 640, 1001) for o in BOTH[1:]})
