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


def test_rows_that_no_wide_store_fits_count():
    """Pairs end a tile slowly where N is no multiple of 8; with few blocks of K that decides (measured on 2048 x 512 ->
    14335: pairs 46 us, 128-token tiles 43; at 14336 23 and 41)."""
    assert F.pick(2048, 14336, 512, 152, PLENTY) == (0, 1)
    assert F.pick(2048, 14335, 512, 152, PLENTY) == (128, 1)
    assert F.pick(512, 6143, 2048, 152, PLENTY) == (0, 1)  # 15.9 and 18.1
    assert F.pick(4096, 2047, 1024, 152, PLENTY) == (0, 1)  # 20.9 and 21.5
