"""CPU test of the numbers that the binding of eviction hands to the C ABI, whose int has 32 bits."""
import ctypes

import pytest

torch = pytest.importorskip("torch")


def test_more_recent_tokens_than_an_int_holds(wql_lib, monkeypatch):
    lib, calls = wql_lib._lib, []
    monkeypatch.setattr(lib, "_is", lambda *a: True)
    monkeypatch.setattr(lib, "_run", lambda fn, index, *a: calls.append([ctypes.c_int(a[i]).value for i in (12, 13)]))
    z = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    for D in (64, 128):
        cache = torch.zeros((2, 2, 1, 16 * (D + 8)), dtype=torch.uint8)
        monkeypatch.setattr(lib, "_cache_dims", lambda c: (2, 2, 16, D))
        for recent in (0, 5, 8, 9, 2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 32 + 3, 2 ** 40):
            wql_lib.kv_evict_i4(torch.zeros((2, 2, 16)), cache, z(2, 1), z(2), z(2, 1), 8, recent)
            budget, got = calls.pop()
            assert budget == 8 and min(got, 8) == min(recent, 8)
        for recent in (-1, -2 ** 31, -2 ** 32, -2 ** 32 + 3):
            with pytest.raises(ValueError, match="recent"):
                wql_lib.kv_evict_i4(torch.zeros((2, 2, 16)), cache, z(2, 1), z(2), z(2, 1), 8, recent)
    assert not calls
