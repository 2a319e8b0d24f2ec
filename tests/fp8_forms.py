"""Calls of the 8-bit products for each form of the launch plan (csrc/mlora_fp8_plan.h):
test_fp8_plan.py keeps them to their forms, test_gpu_fp8_forms.py runs them."""
from __future__ import annotations

NAMES = ("stream", "32 rows", "64 rows", "128 rows", "256 rows")

# experts (0: one weight), n_out, k_in, rows, the form with fp32 sums and with fast ones.
# Five blocks of k and more, so that each stage of LDS is filled again; ragged widths.
FORMS = [
    (0, 300, 640, 60, "stream", "stream"),
    (5, 301, 650, 60, "stream", "stream"),
    (0, 1601, 640, 500, "32 rows", "32 rows"),
    (40, 330, 700, 800, "32 rows", "32 rows"),
    (0, 1300, 640, 2300, "64 rows", "64 rows"),
    (40, 1030, 645, 1400, "64 rows", "64 rows"),
    (0, 2500, 640, 3500, "128 rows", "128 rows"),
    (10, 3300, 641, 2100, "128 rows", "128 rows"),
    (20, 2101, 640, 1600, "64 rows", "128 rows"),
    (0, 2601, 640, 5100, "128 rows", "256 rows"),
    (24, 2050, 650, 3120, "64 rows", "256 rows"),
    (25, 2500, 1290, 5200, "128 rows", "256 rows"),
]
