"""A shape for each launch form of sgemm_w4: the form, rows of X, rows of the
weight (neither whole tiles, more than one tile row or column where the form has
tiles, first and last row counts of a form)."""
SHAPES = [
    (0, 1, 257), (0, 16, 6368), (1, 3, 6369), (1, 16, 12736), (2, 5, 12737), (2, 16, 13001),
    (3, 17, 300), (3, 64, 3137), (3, 65, 1003), (4, 40, 3201), (4, 64, 6272), (5, 33, 6337), (5, 64, 7003), (5, 90, 6499), (5, 128, 8192),
    (6, 65, 11401), (6, 129, 6849), (6, 200, 5003), (7, 300, 12801), (7, 1030, 4001), (7, 128, 31001),
]
FORMS = range(8)
