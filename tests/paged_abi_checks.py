"""Host-side argument checks of the resident paged cache's entry points,
against a bare ctypes handle (see abi_checks.py, whose loader this uses):

    python tests/paged_abi_checks.py PATH_TO_LIBRARY

Every call here fails validation, or has nothing to do, before any HIP call.
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import abi_checks  # noqa: E402

FAKE = abi_checks.FAKE
NAN = float('nan')


def check_paged_append(lib):
    def call(pool=FAKE, slots=1000, rb=1152, ps=16, table=FAKE, ld=10, row0=FAKE, n=FAKE, B=2, T=3, rows=FAKE, rs=1152):
        return lib.ech_paged_append(pool, slots, rb, ps, table, ld, row0, n, B, T, rows, rs, None, None)
    for bad in (dict(pool=None), dict(table=None), dict(row0=None), dict(n=None), dict(rows=None), dict(slots=0),
                dict(slots=1 << 31), dict(rb=0), dict(rb=1150), dict(rs=1136), dict(rs=1160), dict(ps=0),
                dict(ps=(1 << 20) + 1), dict(ld=0), dict(B=0), dict(B=65536), dict(T=-1), dict(pool=FAKE + 8),
                dict(rows=FAKE + 2), dict(rb=(1 << 20) + 16, rs=1 << 21)):
        assert call(**bad) == -1, bad
    assert call(T=0) == 0 and call(T=0, rows=None) == 0


def check_paged_attn(lib):
    assert lib.ech_paged_attn_ws_bytes(0, 1, 16, 1, 10, 0, 0) == 0
    assert lib.ech_paged_attn_ws_bytes(1, 1, 129, 1, 10, 0, 0) == 0
    need = lib.ech_paged_attn_ws_bytes(1, 1, 16, 1, 100000, 0, 0)
    assert need > 0
    big = lib.ech_paged_attn_ws_bytes(1, 4, 16, 4, 100000, 0, 0)
    assert big > need

    def call(q=FAKE, rs=576 * 16, hs=576, pool=FAKE, slots=1000, ps=16, table=FAKE, ld=10, row0=FAKE, n=FAKE, B=1, T=1,
             H=16, mr=1, ml=100000, w=0, sk=0, sc=0.1, out=FAKE, lse=FAKE, ws=FAKE, wb=need):
        return lib.ech_paged_attn(q, rs, hs, pool, slots, ps, table, ld, row0, n, B, T, H, mr, ml, w, sk, sc, out, lse,
                                  ws, wb, None)
    for bad in (dict(q=None), dict(pool=None), dict(table=None), dict(row0=None), dict(n=None), dict(out=None),
                dict(rs=-8), dict(rs=4), dict(hs=577), dict(hs=-576), dict(slots=0), dict(slots=1 << 31), dict(ps=0),
                dict(ld=0), dict(B=0), dict(B=65536), dict(T=-1), dict(H=0), dict(H=129), dict(mr=-1), dict(ml=-1),
                dict(w=-1), dict(sk=-1), dict(sc=NAN), dict(q=FAKE + 2), dict(pool=FAKE + 8), dict(out=FAKE + 4),
                dict(ws=None), dict(ws=FAKE + 16), dict(wb=need - 1), dict(T=1 << 28, mr=1 << 28)):
        assert call(**bad) == -1, bad
    assert call(T=0, mr=0, q=None, out=None, ws=None, wb=0) == 0
    assert call(mr=0, wb=1 << 40) == 0


def check_paged_weight(lib):
    assert lib.ech_paged_weight_ws_bytes(0, 1, 16, 1, 10) == 0
    need = lib.ech_paged_weight_ws_bytes(1, 512, 128, 512, 200)

    def call(q=FAKE, rs=576 * 128, hs=576, lse=FAKE, pool=FAKE, slots=1000, ps=16, table=FAKE, ld=20, row0=FAKE, n=FAKE,
             B=1, T=512, H=128, mr=512, ml=200, w=0, sk=0, sc=0.1, ai=FAKE, ao=FAKE, ald=200, dec=1.0, ws=FAKE,
             wb=need):
        return lib.ech_paged_weight(q, rs, hs, lse, pool, slots, ps, table, ld, row0, n, B, T, H, mr, ml, w, sk, sc, ai,
                                    ao, ald, dec, ws, wb, None)
    for bad in (dict(q=None), dict(lse=None), dict(pool=None), dict(table=None), dict(row0=None), dict(n=None),
                dict(ao=None), dict(ald=199), dict(dec=NAN), dict(sc=NAN), dict(H=0), dict(H=129), dict(w=-1),
                dict(sk=-1), dict(q=FAKE + 8), dict(pool=FAKE + 8), dict(rs=3), dict(hs=-8), dict(B=0), dict(ml=-1),
                dict(slots=0), dict(ps=0), dict(ld=0)):
        assert call(**bad) == -1, bad
    if need:
        assert call(wb=need - 1) == -1 and call(ws=None) == -1 and call(ws=FAKE + 64) == -1
    assert call(ml=0, wb=1 << 40) == 0


def check_paged_evict(lib):
    need = lib.ech_paged_evict_ws_bytes(2, 100000, 500)

    def call(acc=FAKE, ald=100000, n=FAKE, B=2, ml=100000, keep=500, sk=4, rc=16, kept=FAKE, ao=FAKE, lo=FAKE, pool=FAKE,
             slots=1000, rb=1152, ps=16, src=FAKE, dst=FAKE, ld=10, ws=FAKE, wb=need):
        return lib.ech_paged_evict(acc, ald, n, B, ml, keep, sk, rc, kept, ao, lo, pool, slots, rb, ps, src, dst, ld, ws,
                                   wb, None)
    for bad in (dict(acc=None), dict(n=None), dict(kept=None), dict(lo=None), dict(ald=99999), dict(B=0),
                dict(B=65536), dict(ml=-1), dict(keep=0), dict(sk=-1), dict(rc=-1), dict(sk=400, rc=101),
                dict(sk=2 ** 31 - 1, rc=2 ** 31 - 1), dict(slots=0), dict(rb=0), dict(rb=24), dict(ps=0),
                dict(src=None), dict(dst=None), dict(ld=0), dict(pool=FAKE + 8)):
        assert call(**bad) == -1, bad
    if need:
        assert call(wb=need - 1) == -1 and call(ws=None) == -1 and call(ws=FAKE + 64) == -1


CHECKS = [v for k, v in sorted(globals().items()) if k.startswith('check_')]

if __name__ == '__main__':
    lib = abi_checks.load(sys.argv[1])
    for fn in CHECKS:
        fn(lib)
    print(f'paged abi checks ok: {len(CHECKS)}', flush=True)
