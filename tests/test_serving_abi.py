"""CPU checks of the calls around the packed cache: bad arguments are refused before anything touches a device, and the
binding's structs are the C compiler's."""
import ctypes

import pytest

import decode_attention_13_b200 as gtq
from decode_attention_13_b200 import binding

INV, UNS = gtq.GTQ_ERR_INVALID, gtq.GTQ_ERR_UNSUPPORTED
P = 0x1000   # an aligned address that is never followed


def _rope(**kw):
    base = dict(head_dim=128, theta=1e4)
    base.update(kw)
    return gtq.make_rope(base.pop("head_dim"), base.pop("theta"), **base)


def _tensor(**kw):
    t = binding.gtq_rope_tensor(P, P, 2, 0)
    t.x_strides = t.y_strides = (ctypes.c_int64 * 4)(1024, 512, 128, 1)
    for k, v in kw.items():
        setattr(t, k, v)
    return t


def _strides(*s):
    return (ctypes.c_int64 * len(s))(*s)


def _call_rope(cfg, q, batch=1, tokens=4, pos=None, pos_stride=0):
    lib = binding.library()
    return lib.gtq_rope(None if cfg is None else ctypes.byref(cfg), batch, tokens, pos, pos_stride, 0,
                        None if q is None else ctypes.byref(q), None, None)


@pytest.mark.parametrize("kw", [
    dict(head_dim=0), dict(head_dim=127), dict(head_dim=258), dict(rotary_dim=0), dict(rotary_dim=129),
    dict(rotary_dim=130), dict(rope_pairing=2), dict(dtype=2), dict(scaling=4), dict(scaling=-1), dict(theta=1.0),
    dict(theta=float("nan")), dict(theta=float("inf")), dict(magnitude=float("nan")),
    dict(scaling=1, factor=0.5), dict(scaling=1, factor=float("inf")), dict(scaling=2, factor=2.0),
    dict(scaling=2, factor=2.0, original_context=8192, low_freq=4.0, high_freq=4.0),
    dict(scaling=3, factor=2.0, original_context=8192, low_freq=0.0, high_freq=4.0),
    dict(scaling=3, factor=2.0, original_context=8192, low_freq=1.0, high_freq=float("inf")),
])
def test_rope_refuses_bad_configs(kw):
    assert _call_rope(_rope(**kw), _tensor()) == INV


def test_rope_refuses_bad_calls():
    c = _rope()
    assert _call_rope(None, _tensor()) == INV
    assert _call_rope(c, None) == INV
    for t in (_tensor(x=None), _tensor(y=None), _tensor(x=P + 1), _tensor(heads=0), _tensor(heads=65536),
              _tensor(reserved=1), _tensor(x_strides=_strides(0, 0, 128, 2)), _tensor(y_strides=_strides(0, 0, -1, 1))):
        assert _call_rope(c, t) == INV
    assert _call_rope(c, _tensor(), batch=0) == INV
    assert _call_rope(c, _tensor(), tokens=0) == INV
    assert _call_rope(c, _tensor(), pos=P + 4) == INV
    assert _call_rope(c, _tensor(), pos=P, pos_stride=-1) == INV
    assert _call_rope(c, _tensor(), batch=1 << 16, tokens=1 << 16) == UNS
    assert _call_rope(c, _tensor(), batch=1 << 62, tokens=1 << 62) == UNS
    bad = _rope()
    bad.backward = 2
    assert _call_rope(bad, _tensor()) == INV


def test_rope_refuses_rows_that_overlap():
    c = _rope()
    # one row of y for several of x, and in place with another order of dims
    assert _call_rope(c, _tensor(y=2 * P, y_strides=_strides(0, 512, 128, 1)), batch=2) == INV
    assert _call_rope(c, _tensor(y=2 * P, y_strides=_strides(1024, 0, 128, 1))) == INV
    assert _call_rope(c, _tensor(y=2 * P, y_strides=_strides(1024, 512, 0, 1))) == INV
    assert _call_rope(c, _tensor(y_strides=_strides(1024, 128, 256, 1))) == INV


def test_calls_without_a_plan():
    lib = binding.library()
    ch = binding.gtq_chunk(1, None, 1, 0, _strides(0, 128, 0, 1), _strides(0, 128, 0, 1))
    ev = binding.gtq_eviction()
    assert lib.gtq_chunk_attn(None, P, 1, None, ctypes.byref(ch), P, P, P, 1 << 20, None) == INV
    assert lib.gtq_attn_weights(None, P, 1, None, ctypes.byref(ch), P, None, P, _strides(0, 0), P, 1 << 20, None) == INV
    assert lib.gtq_evict(None, P, 1, None, ctypes.byref(ev), P, 1 << 20, None, P, 1 << 20, None) == INV
    assert lib.gtq_chunk_workspace_bytes(None, 1, 1) == 0
    assert lib.gtq_weights_workspace_bytes(None, 1, 1) == 0
    assert lib.gtq_evict_workspace_bytes(None, 1) == 0


def test_struct_layouts_match_the_header(tmp_path):
    import os
    import shutil
    import subprocess

    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    names = ("gtq_rope_config", "gtq_rope_tensor", "gtq_chunk", "gtq_eviction")
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "gtq.h"', 'int main(void) {']
    for n in names:
        lines.append('printf("%s %%zu\\n", sizeof(%s));' % (n, n))
        for f, _ in getattr(binding, n)._fields_:
            lines.append('printf("%s.%s %%zu\\n", offsetof(%s, %s));' % (n, f, n, f))
    lines += ['return 0;', '}']
    (tmp_path / "t.c").write_text("\n".join(lines))
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([cc, "-I", os.path.join(root, "include"), str(tmp_path / "t.c"), "-o", str(tmp_path / "t")], check=True)
    out = subprocess.run([str(tmp_path / "t")], capture_output=True, text=True, check=True).stdout
    got = dict(line.split() for line in out.split("\n") if line)
    for n in names:
        cls = getattr(binding, n)
        assert int(got[n]) == ctypes.sizeof(cls), n
        for f, _ in cls._fields_:
            assert int(got["%s.%s" % (n, f)]) == getattr(cls, f).offset, (n, f)
