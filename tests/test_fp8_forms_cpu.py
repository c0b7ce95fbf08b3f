"""How the e4m3 linear picks its form, without a GPU."""
import os
import subprocess

import fp8_forms as F

HERE = os.path.dirname(os.path.abspath(__file__))
PLENTY = lambda tn, split: 152 // split  # noqa: E731


def test_answers_are_kept_per_device(tmp_path):
    exe = tmp_path / "memo"
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Wextra", "-Werror", os.path.join(HERE, "device_memo.cc"), "-o", str(exe)],
                   check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.stdout + out.stderr


def test_a_failed_query_fails_the_call():
    """Rather than picking an unsplit form, which sums in another order than the same call's next one."""
    failing = lambda tn, split: -2 if split == 8 else 152 // split  # noqa: E731
    assert F.pick(1, 1024, 6144, 152, PLENTY) == (16, 8)
    assert F.pick(1, 1024, 6144, 152, failing) == (-1, -2)
    assert F.pick(8192, 14336, 4096, 152, failing) == (0, 1)  # no cluster is asked about: no split fits


def test_a_split_keeps_to_the_clusters_that_run_at_once():
    for most in (19, 12, 8, 7, 1, 0):
        tn, split = F.pick(1, 1024, 6144, 152, lambda t, s, most=most: most if s == 8 else 152 // s)
        assert (tn, split) == ((16, 8) if most >= 8 else (16, 4))  # 8 tiles of 128 weight rows
