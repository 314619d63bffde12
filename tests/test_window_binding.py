"""What the binding hands to the library as C ints (a stand-in for the library, CPU tensors: nothing is launched)."""

import ctypes

import pytest

torch = pytest.importorskip("torch")

from exact_tiled_attention_07_gb300 import binding as fa  # noqa: E402

TOP = 2 ** 31 - 1


class Library:
    """Takes down what a call gets, ints as ctypes hands them over."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, [ctypes.c_int(a).value if type(a) is int else a for a in args]))
            return 0 if not name.endswith("workspace_size") else 64
        return call


@pytest.fixture
def lib(monkeypatch):
    lib = Library()
    monkeypatch.setattr(fa, "load_library", lambda path=None: lib)
    monkeypatch.setattr(fa, "_ready", lambda *ts, strided=(): None)
    monkeypatch.setattr(fa, "_on_device", lambda *ts, strided=(): None)
    monkeypatch.setattr(fa, "_stream", lambda stream: 0)
    monkeypatch.setattr(fa, "_current", lambda stream: 0)
    return lib


def calls(fa):
    q, k, lse = torch.zeros(1, 4, 6, 64).half(), torch.zeros(1, 2, 6, 64).half(), torch.zeros(1, 4, 6)
    p, pk, cu = torch.zeros(6, 4, 64).half(), torch.zeros(6, 2, 64).half(), torch.tensor([0, 6], dtype=torch.int32)
    lens, ws = torch.tensor([6], dtype=torch.int32), torch.zeros(64, dtype=torch.uint8)
    return {
        "fa_fwd_window": (lambda w, s: fa.fa_fwd_window(q, k, k, q, lse, 1.0, w, s), "fa_fwd_window"),
        "fa_bwd_window": (lambda w, s: fa.fa_bwd_window(q, k, k, q, q, lse, q, k, k, ws, 1.0, w, s), "fa_bwd_window"),
        "fa_fwd_varlen_window": (lambda w, s: fa.fa_fwd_varlen_window(p, pk, pk, p, lse, cu, 1.0, w, s), "fa_fwd_varlen_window"),
        "fa_decode_window": (lambda w, s: fa.fa_decode_window(q, k, k, lens, q, lse, 1.0, w, s, ws), "fa_decode_window"),
        "attention_forward": (lambda w, s: fa.attention_forward(q, k, k, causal=True, window=w, sinks=s), "fa_fwd_window"),
        "attention_backward": (lambda w, s: fa.attention_backward(q, k, k, q, q, lse, causal=True, window=w, sinks=s, workspace=ws),
                               "fa_bwd_window"),
        "attention_decode_window": (lambda w, s: fa.attention_decode_window(q, k, k, lens, w, s), "fa_decode_window"),
        "attention_forward_varlen": (lambda w, s: fa.attention_forward_varlen(p, pk, pk, cu, causal=True, window=w, sinks=s),
                                     "fa_fwd_varlen_window"),
    }


@pytest.mark.parametrize("name", list(calls(fa)))
@pytest.mark.parametrize("big", [2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 40])
def test_windows_and_sinks_past_an_int_are_the_largest(lib, name, big):
    call, entry = calls(fa)[name]

    def pair():  # (window and sinks stand side by side in every call's arguments, the window in front)
        args = [args for n, args in lib.calls if n == entry][-1]
        at = next(i for i, a in enumerate(args) if type(a) is float) + 1  # behind the scale
        return args[at:at + 2]

    call(TOP, 4)
    assert pair() == [TOP, 4]
    call(big, 4)
    assert pair() == [TOP, 4]
    call(7, big)
    assert pair() == [7, TOP]


def test_a_window_without_sinks_past_an_int(lib):
    q, lse = torch.zeros(1, 4, 6, 64).half(), torch.zeros(1, 4, 6)
    fa.fa_fwd_masked(q, q, q, q, lse, 1.0, True, window=2 ** 32 + 5)
    name, args = lib.calls[-1]
    assert name == "fa_fwd_masked" and TOP in args and 5 not in args
