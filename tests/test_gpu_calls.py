"""The ways an operator's call takes: its quick form, the form in Python, ctypes; all
give the same, refuse the same, and may be taken by several threads at once."""
import threading

import numpy as np
import pytest
import torch

import slots4_testlib as four
import slots_testlib as plain

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import kv_cache_compression_c128_gb300 as kvc

    kvc.build()
    kvc._load_torch()
    if kvc._quick is None:
        pytest.skip("built without the interpreter's or torch's headers")
    return kvc


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _arguments(seed=0):
    rng = np.random.default_rng(seed)
    R, H, lengths = 3, 20, [200, 0, 65]
    table, pool = plain.page_tables(rng, lengths)
    kv = cuda(four.random_cache(rng, pool))
    x = cuda(rng.standard_normal((9, 512)).astype(np.float32))
    slots = cuda(rng.permutation(64 * pool)[:9].astype(np.int64))
    turns = cuda(four.table_of(300))
    positions = cuda(rng.integers(0, 300, (9, 2)))
    names = bytes([0] * 20 + [1] * 12)
    q = cuda(rng.standard_normal((9, H, 512)).astype(np.float32)).to(torch.bfloat16)
    return dict(R=R, H=H, kv=kv, table=cuda(table), lengths=cuda(np.array(lengths, np.int32)), x=x, slots=slots, turns=turns,
                positions=positions, names=names, q=q, sinks=cuda(rng.standard_normal(H).astype(np.float32)))


def _everything(kvc, a):
    """Every operator once, with results given where they can be."""
    R, H = a["R"], a["H"]
    kv = a["kv"].clone()
    assert kvc.store(a["x"], kv, a["slots"], positions=a["positions"], cos_sin_cache=a["turns"], axes=a["names"]) is kv
    kvc.store(a["x"][:1].to(torch.bfloat16), kv, a["slots"][:1])
    back = torch.empty((9, 512), dtype=torch.bfloat16, device="cuda")
    assert kvc.dequantize(kv, a["slots"], torch.bfloat16, out=back) is back
    rows = torch.zeros_like(a["q"])
    view = rows[..., 448:]
    assert kvc.rotate(a["q"][..., 448:], a["positions"], a["turns"], axes=a["names"], inverse=True, out=view) is view
    one = kvc.rotate(a["q"][:, 0, 448:], a["positions"][:, 0], a["turns"], out=torch.empty((9, 64), dtype=torch.bfloat16, device="cuda"))
    out, lse = torch.empty((R, H, 512), dtype=torch.bfloat16, device="cuda"), torch.empty((R, H), device="cuda")
    weights = torch.full((R, 256), 0.5, device="cuda")
    space = torch.empty(kvc.kvc_attend_workspace_bytes(R, H, a["table"].shape[1], True), dtype=torch.uint8, device="cuda")
    got = kvc.attend(a["q"][:R], kv, a["table"], a["lengths"], 0.05, sinks=a["sinks"], out=out, lse=lse, slot_weights=weights,
                     slot_weights_in=weights, workspace=space)
    assert got[0] is out and got[1] is lse
    more = kvc.attend(a["q"][:R], kv, a["table"], a["lengths"], out=out.clone(), lse=lse.clone(), workspace=space)
    return [kv, back, rows, one, out, lse, weights, *more]


def test_every_way_gives_the_same(kvc, monkeypatch):
    a = _arguments()
    want = _everything(kvc, a)
    monkeypatch.setattr(kvc, "_quick", None)
    assert kvc._entry() is kvc.lib()
    for g, w in zip(_everything(kvc, a), want):
        assert torch.equal(g, w)


def test_the_quick_forms_are_taken(kvc, monkeypatch):
    # with the C library's answers in their place, no argument of _everything falls to the other form
    a = _arguments()
    asked = []

    class Asked:
        def __getattr__(self, name):
            f = getattr(kvc_quick, name)

            def call(*args):
                st = f(*args)
                asked.append((name, st))
                return st

            return call

    kvc_quick = kvc._quick
    monkeypatch.setattr(kvc, "_quick", Asked())
    _everything(kvc, a)
    assert [st for name, st in asked if not name.startswith("kvc_")] == [0] * 7
    assert not [name for name, st in asked if name.startswith("kvc_")]


def test_what_is_not_plainly_right_is_left_to_the_other_form(kvc):
    a, quick = _arguments(), kvc._quick
    f32 = torch.empty((9, 512), device="cuda")
    for x, kv, slots, p, t, axes in [
            (a["x"].half(), a["kv"], a["slots"], None, None, None), (a["x"], a["kv"][:, :-1], a["slots"], None, None, None),
            (a["x"], a["kv"].cpu(), a["slots"], None, None, None), (a["x"], a["kv"], a["slots"].int(), None, None, None),
            (a["x"], a["kv"], a["slots"][:8], None, None, None), (a["x"][:0], a["kv"], a["slots"][:0], None, None, None),
            (a["x"], a["kv"], a["slots"], a["positions"], a["turns"], None), (a["x"], a["kv"], a["slots"], None, a["turns"], None),
            (a["x"], a["kv"], a["slots"], a["positions"], a["turns"], bytes([2] * 32)),
            (a["x"], a["kv"], a["slots"], a["positions"], a["turns"], list(a["names"])),
            (a["x"], a["kv"], a["slots"], a["positions"], a["turns"][:, :32], a["names"]),
            (None, None, None, None, None, None), (1, "x", a, a, a, a)]:
        assert quick.store(x, kv, slots, p, t, axes) is None
    for args in [(a["kv"], a["slots"], f32[:8]), (a["kv"], a["slots"], f32.double()), (a["kv"], a["slots"], f32.cpu()),
                 (a["kv"][:, :64], a["slots"], f32), (a["kv"], [1], f32), (a["kv"], a["slots"], None)]:
        assert quick.dequantize(*args) is None
    x = torch.empty((9, 2, 64), device="cuda")
    for args in [(x, a["positions"], a["turns"], None, False, x), (x, a["positions"], a["turns"], a["names"], False, x[:8]),
                 (x.transpose(1, 2), a["positions"], a["turns"], a["names"], False, x), (x, a["positions"].int(), a["turns"], a["names"], False, x),
                 (x[..., :32], a["positions"], a["turns"], a["names"], False, x[..., :32]), (x, a["positions"], a["turns"], a["names"], False, None)]:
        assert quick.rotate(*args) is None
    with pytest.raises(TypeError):
        quick.rotate(x)
    with pytest.raises(TypeError):
        quick.kvc_rotate(1, 2, 3)
    for wrong in ({"slots": a["slots"].int()}, {"x": a["x"].half()}):
        with pytest.raises(TypeError):
            kvc.store(**dict(dict(x=a["x"], kv_cache=a["kv"], slots=a["slots"]), **wrong))
    with pytest.raises(kvc.KvcError):
        kvc.rotate(x, a["positions"], a["turns"][:0], axes=a["names"], out=x)


def test_several_threads_at_once(kvc):
    a = _arguments()
    want = _everything(kvc, a)
    torch.cuda.synchronize()
    wrong = []

    def work():
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(30):
                    got = _everything(kvc, a)
                    torch.cuda.current_stream().synchronize()
                    if not all(torch.equal(g, w) for g, w in zip(got, want)):
                        wrong.append("another result")
        except Exception as e:  # noqa: BLE001 (told by the thread that waits)
            wrong.append(e)

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    assert kvc.kvc_get_device_error(torch.cuda.current_stream().cuda_stream) == 0
