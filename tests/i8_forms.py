"""Sizes of matmul_i8 that each of its forms runs, in place and with fragments moved: what
test_i8_plan.py asserts on the host, and test_gpu_i8_forms.py runs.

(form, moved, M, N, K, pad, off): rows of a and w lie K + pad bytes apart and begin `off` bytes behind
a whole line.  For each form and either way: reductions of whole stages, and ones that end inside a
stage at a multiple of 16, of 4 and at an odd byte.  Rows and columns end inside a tile, columns
inside a store."""
FORMS = [
    ("16x16", False, 3, 109, 2352, 0, 0),
    ("16x16", False, 3, 125, 2584, 0, 0),
    ("16x16", False, 3, 106, 2309, 3, 0),
    ("16x16", False, 3, 117, 2304, 0, 0),
    ("16x16", True, 3, 113, 2320, 0, 3),
    ("16x16", True, 3, 142, 2581, 0, 3),
    ("16x16", True, 3, 134, 2304, 1, 0),
    ("16x16", False, 50, 250, 1044, 0, 0),
    ("16x16", True, 45, 301, 1001, 0, 0),
    ("32x32", False, 17, 2529, 2384, 0, 0),
    ("32x32", False, 18, 4253, 1028, 0, 0),
    ("32x32", False, 17, 4217, 1033, 3, 0),
    ("32x32", False, 18, 2230, 2048, 0, 0),
    ("32x32", True, 17, 2149, 1040, 0, 3),
    ("32x32", True, 17, 2299, 1073, 0, 1),
    ("32x32", True, 17, 2335, 2048, 1, 0),
    ("32x64", False, 18, 8301, 1040, 0, 0),
    ("32x64", False, 17, 8311, 1084, 0, 0),
    ("32x64", False, 17, 8635, 1029, 3, 0),
    ("32x64", False, 34, 4122, 1024, 0, 0),
    ("32x64", True, 33, 4105, 1040, 0, 2),
    ("32x64", True, 17, 8474, 1033, 0, 3),
    ("32x64", True, 33, 4141, 1024, 3, 3),
    ("128x64", False, 132, 6595, 1056, 0, 0),
    ("128x64", False, 4168, 198, 1032, 0, 0),
    ("128x64", False, 3274, 259, 1033, 3, 0),
    ("128x64", False, 2052, 201, 1024, 0, 0),
    ("128x64", True, 4175, 193, 1040, 0, 1),
    ("128x64", True, 4143, 202, 1089, 0, 3),
    ("128x64", True, 2758, 323, 1024, 3, 3),
    ("128x128 deep", False, 130, 8713, 1056, 0, 0),
    ("128x128 deep", False, 130, 8673, 1076, 0, 0),
    ("128x128 deep", False, 141, 8238, 1033, 3, 0),
    ("128x128 deep", False, 135, 8230, 1024, 0, 0),
    ("128x128", False, 399, 8214, 1040, 0, 0),
    ("128x128", False, 408, 8198, 1044, 0, 0),
    ("128x128", False, 399, 8429, 1029, 3, 0),
    ("128x128", False, 514, 6543, 1024, 0, 0),
    ("128x128", True, 162, 8411, 1040, 0, 2),
    ("128x128", True, 161, 8790, 1059, 0, 3),
    ("128x128", True, 162, 8221, 1024, 1, 2),
    ("192x256", False, 921, 8243, 1056, 0, 0),
    ("192x256", False, 1034, 7593, 1032, 0, 0),
    ("192x256", False, 1170, 6597, 1029, 3, 0),
    ("192x256", False, 917, 8350, 1024, 0, 0),
    ("192x256", True, 1418, 5433, 1040, 0, 1),
    ("192x256", True, 1422, 5434, 1029, 0, 3),
    ("192x256", True, 914, 8250, 1024, 1, 0),
    ("256x256", False, 1765, 6449, 1040, 0, 0),
    ("256x256", False, 1353, 8265, 1036, 0, 0),
    ("256x256", False, 2314, 4887, 1033, 3, 0),
    ("256x256", False, 1362, 8271, 1024, 0, 0),
    ("256x256", True, 4038, 2825, 1040, 0, 1),
    ("256x256", True, 1751, 6446, 1027, 0, 1),
    ("256x256", True, 1571, 7218, 1024, 3, 2),
]
# (M, N, K) whose last rows go into a launch of their own, and the forms of the two
TWO = [
    (4101, 4003, 1536, "256x256", "16x16"),
    (4097, 12282, 2064, "256x256", "16x16"),
    (2205, 7738, 1044, "256x256", "128x64"),
    (2050, 7305, 1537, "256x256", "16x16"),
    (1048, 3650, 1537, "128x128", "32x32"),
    (2309, 1669, 2048, "128x128 deep", "16x16"),
]


def name(case):
    form, moved, M, N, K, pad, off = case
    return f"{form.replace(' ', '_')}-{'moved' if moved else 'in_place'}-{M}x{N}x{K}" + (f"+{pad}" if pad else "") + (f"@{off}" if off else "")
