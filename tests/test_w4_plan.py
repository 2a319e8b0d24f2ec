"""The launch plan of the 4-bit products (csrc/mlora_w4_plan.h, host code of sizes
alone): every form that a call can be given has a case in w4_cases.FORMS, which
the GPU tests run, and each case there is given the form it stands for."""
from __future__ import annotations

import math
import os
import random
import shutil
import subprocess

import pytest

from tests.w4_cases import FORMS

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
FIELDS = ("stream", "by_row", "places", "mb", "tiles", "waves", "k_waves", "splits", "per_slice",
          "slices", "panels")


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    exe = str(tmp_path_factory.mktemp("plan") / "w4_plan")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "include"), "-I",
                    os.path.join(ROOT, "moe_expert_lora_amd", "csrc"),
                    os.path.join(HERE, "w4_plan.cpp"), "-o", exe], check=True, timeout=120)

    def run(calls):
        text = "\n".join(" ".join(map(str, c)) for c in calls)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True,
                             timeout=60)
        return [dict(zip(FIELDS, map(int, line.split()))) for line in out.stdout.splitlines()]
    return run


def _form(p):
    waves = p["waves"] // p["k_waves"]
    parts = ["stream" if p["stream"] else "split", f"mb{p['mb']}"]
    if p["stream"]:
        parts += [f"kw{p['k_waves']}", "pairs" if p["per_slice"] > waves else "",
                  "panels" if p["panels"] else ""]
    else:
        parts.append(f"tiles{p['tiles']}")
    parts += ["byrow" if p["by_row"] else "", "splits" if p["splits"] > 1 else ""]
    return " ".join(x for x in parts if x)


def test_cases_have_their_forms(plans):
    got = plans([c[:6] for c in FORMS])
    for case, p in zip(FORMS, got):
        assert _form(p) == case[6], (case, p)


def test_every_form_has_a_case(plans):
    """Over a seeded sweep of the sizes that calls have."""
    rng = random.Random(1)
    log = lambda a, b: int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))  # noqa: E731
    calls = []
    for _ in range(100000):
        experts = rng.choice([0, 0, log(2, 1024), log(2, 300)])
        calls.append((log(1, 40000 if experts else 5000), experts, log(1, 1024) * 8, log(1, 20000),
                      rng.choice([32, 64, 128, 256]), rng.randrange(2)))
    have = {(c[6], c[5]) for c in FORMS}
    for call, p in zip(calls, plans(calls)):
        assert (_form(p), call[5]) in have, (call, p)


def test_what_a_plan_must_keep(plans):
    """Workgroups cover every column pair once and hold at most 12 waves; sums that
    stay in registers (several panels, or several waves to a pair) are of one pair a
    wave, which the kernels take for granted."""
    rng = random.Random(2)
    log = lambda a, b: int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))  # noqa: E731
    calls = [(log(1, 1 << 30 if e == 0 else 1 << 20), e, log(1, 1 << 17) * 8, log(1, 1 << 20),
              rng.choice([32, 64, 128, 1280]), rng.randrange(2))
             for e in (rng.choice([0, 1, 1024, log(1, 1024)]) for _ in range(50000))]
    for c, p in zip(calls, plans(calls)):
        tiles = -(-c[3] // 16)
        assert 1 <= p["waves"] <= 12 and 1 <= p["splits"] <= 32 and p["slices"] <= 1 << 16
        assert p["places"] <= 1024 and p["mb"] in (1, 2) and not (c[5] and p["mb"] == 2)
        if not p["stream"]:
            assert p["waves"] <= 8 and p["tiles"] in (1, 2)
            assert (p["slices"] - 1) * p["tiles"] < tiles <= p["slices"] * p["tiles"]
            assert p["tiles"] == 1 or c[5] or p["mb"] == 2
            continue
        pairs = -(-tiles // 2)
        assert (p["slices"] - 1) * p["per_slice"] < pairs <= p["slices"] * p["per_slice"]
        assert p["waves"] % p["k_waves"] == 0 and 1 <= p["k_waves"] <= 4
        if p["panels"] or p["k_waves"] > 1:
            assert p["per_slice"] <= p["waves"] // p["k_waves"], (c, p)
