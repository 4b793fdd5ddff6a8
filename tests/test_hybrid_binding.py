"""The binding of gdn_hybrid.h on the CPU: what a call hands to the library, seen in place of it."""
import threading

import pytest

A = 0x10000  # an address that is never read


@pytest.fixture
def H(monkeypatch):
    import gated_delta_rule_34_amd as G

    H = G.hybrid
    monkeypatch.setattr(H, "_begin", lambda p, t, name: (0, None))
    monkeypatch.setattr(H, "_rows", lambda *a: (A, 512))
    monkeypatch.setattr(H, "_pages", lambda k, v, *a: (A, A, k, 16))  # (the pool stands for its number of pages)
    monkeypatch.setattr(H, "_on", lambda *a: 0)
    return H


def problem(H):
    p = H.gdn_paged_problem(N=2, Hq=8, Hk=2, D=64, page_size=16, max_pages=5, max_len=80, scale=0.125, page_table=A, lens=A)
    p._any = True  # the pages at the call give their number
    return p


def test_calls_at_once_keep_their_own_pools(H, monkeypatch):
    """Two threads call with one problem and pools of different sizes: each call's pages are checked against its own."""
    p, both, seen = problem(H), threading.Barrier(2, timeout=60), {}

    def call(name, q, *args):
        both.wait()  # both have made their arguments
        seen[threading.current_thread().name] = q.n_pages

    monkeypatch.setattr(H, "_call", call)
    threads = [threading.Thread(target=H.gdn_paged_attn_decode, args=(p, None, n, n, None, None, None), name=str(n)) for n in (3, 700)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert seen == {"3": 3, "700": 700}


def test_a_call_leaves_the_problem_as_it_was(H, monkeypatch):
    p, seen = problem(H), []
    monkeypatch.setattr(H, "_call", lambda name, q, *args: seen.append(bytes(q)))
    before = bytes(p)
    H.gdn_paged_attn_decode(p, None, 10, 10, None, None, None)
    assert bytes(p) == before
    p.n_pages = 10
    assert seen == [bytes(p)]  # all else is the caller's
