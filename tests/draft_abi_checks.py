"""Host-side argument checks of the entry points for drafted tokens, against a
bare ctypes handle (see abi_checks.py, whose loader this uses):

    python tests/draft_abi_checks.py PATH_TO_LIBRARY

Every call here fails validation, or has nothing to do, before any HIP call.
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import abi_checks  # noqa: E402

FAKE = abi_checks.FAKE
NAN = float('nan')


def check_paged_tree_attn(lib):
    size = lib.ech_paged_tree_attn_ws_bytes
    assert size(1, 300, 16, 257, 100000, 0, 0) == 0 and size(0, 1, 16, 1, 10, 0, 0) == 0
    need = size(1, 4, 16, 4, 100000, 0, 0)
    assert need == lib.ech_paged_attn_ws_bytes(1, 4, 16, 4, 100000, 0, 0) > 0

    def call(q=FAKE, rs=576 * 16, hs=576, pool=FAKE, slots=1000, ps=16, table=FAKE, ld=10, row0=FAKE, n=FAKE, par=FAKE,
             B=1, T=4, H=16, mr=4, ml=100000, w=0, sk=0, sc=0.1, out=FAKE, lse=FAKE, ws=FAKE, wb=need):
        return lib.ech_paged_tree_attn(q, rs, hs, pool, slots, ps, table, ld, row0, n, par, B, T, H, mr, ml, w, sk, sc,
                                       out, lse, ws, wb, None)
    for bad in (dict(par=None), dict(mr=257), dict(mr=257, wb=1 << 40), dict(q=None), dict(pool=None), dict(table=None),
                dict(row0=None), dict(n=None), dict(out=None), dict(rs=-8), dict(hs=577), dict(slots=0), dict(ps=0),
                dict(ld=0), dict(B=0), dict(B=65536), dict(T=-1), dict(H=0), dict(H=129), dict(mr=-1), dict(ml=-1),
                dict(w=-1), dict(sk=-1), dict(sc=NAN), dict(q=FAKE + 2), dict(pool=FAKE + 8), dict(out=FAKE + 4),
                dict(ws=None), dict(ws=FAKE + 16), dict(wb=need - 1)):
        assert call(**bad) == -1, bad
    assert call(T=0, mr=0, q=None, out=None, par=None, ws=None, wb=0) == 0
    assert call(mr=0, wb=1 << 40) == 0


def check_draft_verify(lib):
    size = lib.ech_draft_verify_ws_bytes
    assert size(0, 1, 10, 1, 1) == 0 and size(1, 1, 0, 1, 1) == 0 and size(1, 1, 10, 257, 1) == 0
    assert size(1, 1, 10, 1, 0) == 0 and size(1, 1 << 30, 1 << 24, 1, 1) == 0
    need = size(2, 6, 1000, 3, 4)
    assert 0 < need < size(2, 6, 100000, 3, 4)

    def call(x=FAKE, lt=0, ld=1000, V=1000, tok=FAKE, row0=FAKE, par=None, q=None, ldq=1000, u=FAKE, t=FAKE, B=2, T=6,
             mr=3, most=4, kept=FAKE, nk=FAKE, nx=FAKE, ws=FAKE, wb=need):
        return lib.ech_draft_verify(x, lt, ld, V, tok, row0, par, q, ldq, u, t, B, T, mr, most, kept, nk, nx, ws, wb, None)
    for bad in (dict(x=None), dict(ld=999), dict(V=0), dict(V=(1 << 24) + 1, ld=1 << 25), dict(tok=None), dict(row0=None),
                dict(u=None), dict(B=0), dict(B=65536), dict(T=-1), dict(mr=-1), dict(mr=257), dict(most=0),
                dict(kept=None), dict(nk=None), dict(nx=None), dict(ws=None), dict(ws=FAKE + 16), dict(wb=need - 1),
                dict(x=FAKE + 1), dict(lt=1, x=FAKE + 2), dict(q=FAKE, par=FAKE), dict(q=FAKE, ldq=999),
                dict(q=FAKE + 2)):
        assert call(**bad) == -1, bad
    assert call(lt=2) == -3 and call(lt=-1) == -3


def check_paged_accept(lib):
    def call(pool=FAKE, slots=1000, rb=1152, ps=16, table=FAKE, ld=10, row0=FAKE, n=FAKE, B=2, mr=4, ml=100, kept=FAKE,
             most=4, nk=FAKE, lo=FAKE):
        return lib.ech_paged_accept(pool, slots, rb, ps, table, ld, row0, n, B, mr, ml, kept, most, nk, lo, None)
    for bad in (dict(pool=None), dict(table=None), dict(row0=None), dict(n=None), dict(kept=None), dict(nk=None),
                dict(lo=None), dict(slots=0), dict(slots=1 << 31), dict(rb=0), dict(rb=1150), dict(rb=(1 << 20) + 16),
                dict(ps=0), dict(ps=(1 << 20) + 1), dict(ld=0), dict(B=0), dict(B=65536), dict(mr=-1), dict(ml=-1),
                dict(ml=(1 << 30) + 1), dict(most=0), dict(pool=FAKE + 8)):
        assert call(**bad) == -1, bad


def check_paged_copy(lib):
    def call(pool=FAKE, slots=1000, rb=1152, ps=16, src=FAKE, dst=FAKE, rows=None, n=3):
        return lib.ech_paged_copy(pool, slots, rb, ps, src, dst, rows, n, None)
    for bad in (dict(pool=None), dict(src=None), dict(dst=None), dict(slots=0), dict(slots=1 << 31), dict(rb=0),
                dict(rb=8), dict(rb=1160), dict(rb=(1 << 20) + 16), dict(ps=0), dict(ps=(1 << 20) + 1), dict(n=-1),
                dict(pool=FAKE + 4), dict(rb=1 << 20, ps=1 << 20)):
        assert call(**bad) == -1, bad
    assert call(n=0) == 0 and call(n=0, src=None, dst=None) == 0


CHECKS = [v for k, v in sorted(globals().items()) if k.startswith('check_')]

if __name__ == '__main__':
    lib = abi_checks.load(sys.argv[1])
    for fn in CHECKS:
        fn(lib)
    print(f'draft abi checks ok: {len(CHECKS)}', flush=True)
