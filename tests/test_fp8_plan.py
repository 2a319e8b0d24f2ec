"""The launch plan of the 8-bit products (csrc/mlora_fp8_plan.h, host code of sizes
alone): each case of fp8_forms.FORMS has the form that it stands for, and every form
has cases, so that a changed rule does not leave a kernel without a test."""
from __future__ import annotations

import math
import os
import random
import shutil
import subprocess

import pytest

from tests.fp8_forms import FORMS, NAMES

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    exe = str(tmp_path_factory.mktemp("plan") / "fp8_plan")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "moe_expert_lora_amd", "csrc"),
                    os.path.join(HERE, "fp8_plan.cpp"), "-o", exe], check=True, timeout=120)

    def run(calls):
        text = "\n".join(" ".join(map(str, c)) for c in calls)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True,
                             timeout=60)
        return [NAMES[int(line)] for line in out.stdout.split()]
    return run


def test_cases_have_their_forms(plans):
    for fast in (0, 1):
        got = plans([(n, max(E, 1), N, fast) for E, N, K, n, *_ in FORMS])
        assert got == [c[4 + fast] for c in FORMS]


def test_every_form_has_cases(plans):
    """One weight and many, with either kind of sums; the largest tile is of fast ones."""
    for fast in (0, 1):
        for one in (True, False):
            have = {c[4 + fast] for c in FORMS if (c[0] == 0) == one}
            assert have == set(NAMES if fast else NAMES[:4])
    rng = random.Random(1)
    log = lambda a, b: int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))  # noqa: E731
    calls = [(log(1, (1 << 30) - 1), rng.choice([1, log(1, 1024)]), log(1, 1 << 20))
             for _ in range(20000)]
    assert set(plans([(*c, 0) for c in calls])) == set(NAMES[:4])
    assert set(plans([(*c, 1) for c in calls])) == set(NAMES)
