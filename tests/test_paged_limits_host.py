"""Sizes and aliases that the paged-cache entry points refuse on the host, and the extension module that may be missing.  No
GPU needed."""
import importlib.util
import os
import shutil
import subprocess
import sys

import pytest

from test_paged_host import P, SHAPE, attn, kv, ms, rope, verify

L = ms._lib
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_attention_refuses_as_many_tiles_as_its_counts_could_not_pass():
    # 993 sequences of 2162622 tiles of 64 positions are 2^31 - 2: the kernel rounds the count up to whole runs for its CTAs,
    # which has to stay below 2^31 as well
    huge = dict(max_pages=2162622, page_size=64, page_stride=1 << 12, batch=993, n_kv_heads=1)
    assert 993 * 2162622 == 2 ** 31 - 2
    assert attn(kv(**huge), heads=1, ldq=64, ldo=64, most=1, size=1 << 62) == SHAPE
    assert L.ms_op_attn_paged_workspace(kv(**huge), ms.MS_ELEM_F16, 1, 1, 0) == 0


MOST = 1 << 30


def test_rows_and_vocabularies_past_the_kernels_indices_are_refused():
    for n in (MOST + 1, 2 ** 31 - 1):
        assert rope(rows=n) == SHAPE and attn(rows=n) == SHAPE and verify(rows=n) == SHAPE
        assert verify(vocab=n, ldt=1 << 32, ldd=1 << 32) == SHAPE


def test_in_place_needs_the_same_row_stride():
    # another stride would let one row's result overwrite another row's input
    assert rope(out=P, ldo=1024) == SHAPE and "in place" in ms.last_error()
    assert attn(out=P, ldo=1024) == SHAPE and "in place" in ms.last_error()


def _package(tmp_path, extension):
    pkg = tmp_path / "decoder_only_transformer_int4_b200"
    pkg.mkdir()
    src = os.path.join(ROOT, "decoder_only_transformer_int4_b200")
    shutil.copy(os.path.join(src, "__init__.py"), pkg)
    os.symlink(os.path.join(src, "libms_b200.so"), pkg / "libms_b200.so")
    if extension:
        name = [f for f in os.listdir(src) if f.startswith("_paged.") and f.endswith(".so")][0]
        (pkg / name).write_bytes(b"not a library")
    return tmp_path


@pytest.mark.parametrize("extension", [False, True])
def test_the_model_path_works_without_the_extension(tmp_path, extension):
    # the extension belongs to one Python and one torch; what goes through ctypes does not need it
    code = ("import decoder_only_transformer_int4_b200 as ms\n"
            "assert ms._lib.ms_op_status(None, None) == ms.MS_ERR_INVALID_ARG and ms.Model and ms.Cache\n"
            "try:\n    ms.verify_draft(*[None] * 7)\n"
            "except ImportError as e:\n    assert 'build.py' in str(e), e\n    print('said so')\n")
    env = dict(os.environ, PYTHONPATH=str(_package(tmp_path, extension)))
    r = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True, timeout=300, cwd=str(tmp_path))
    assert r.returncode == 0 and "said so" in r.stdout, r.stderr[-2000:]


def test_the_extension_is_built_again_for_another_torch(tmp_path, monkeypatch):
    spec = importlib.util.spec_from_file_location("ms_builder", os.path.join(ROOT, "decoder_only_transformer_int4_b200", "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    b.build()
    assert not b._extension_stale()
    monkeypatch.setattr(b, "_extension_for", lambda: "another torch")
    assert b._extension_stale()
