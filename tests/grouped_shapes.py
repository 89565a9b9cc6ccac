"""Which kernel a grouped product takes, as launch_grouped_product and grouped_vjp choose it, and calls that between them
take every compiled one (tests/test_grouped_dispatch.py compares with the library, tests/test_gpu_grouped_forms.py runs
them)."""

FWD, GX, GXD, PLAIN = 0, 1, 2, 3  # x; grad_y and z; a kept d; grad_y as it is


def product(f32, kind, M, G, KD, ND):
    """('thin' | 'resident' | 'stream', type, kind, ...) of rows with KD entries into ND columns."""
    typ = "float" if f32 else "unsigned short"
    tiles, rows, lies = (M >> 4) + G, M // G, KD <= 128
    if tiles * -(-ND // 64) <= (2048 if lies else 128) or rows < ((64 if f32 else 32) if lies else 48 if f32 else 0):
        return "thin", typ, kind
    if kind != GXD:
        if lies:
            return "resident", typ, kind, -(-KD // 32)
        if ND <= 64:
            return "stream", typ, kind, 2, 32 if ND <= 32 else 64
    return "stream", typ, kind, 4 if f32 and rows >= 4096 else 2, 128


def chunks(n):
    return 1 if n <= 32 else 2 if n <= 64 else 4


def forward(f32, M, G, K, N):
    return {product(f32, FWD, M, G, K, N)}


def vjp(f32, act, M, G, K, N):
    """Of a call that asks for all three gradients."""
    typ, plain = "float" if f32 else "unsigned short", act == "none"
    if K <= 128 and N <= 128:
        return {("panel", typ, chunks(K), chunks(N), plain, False)}
    keeps = K > 128 and N > 128 and not plain
    panel = ("panel", typ, 4, 4, False, True) if keeps else ("panel", typ, chunks(K), chunks(N), plain, False)
    return {panel, product(f32, GXD if keeps else PLAIN if plain else GX, M, G, N, K)}


# rows, groups, inputs, outputs of forward calls
FORWARD = [(300, 3, 60, 70), (40000, 4, 30, 64), (40000, 4, 50, 64), (40000, 4, 80, 64), (40000, 40, 96, 300),
           (40000, 4, 128, 130), (9000, 4, 256, 30), (9000, 4, 200, 64), (9000, 40, 200, 130), (9000, 2, 200, 130)]
# and of VJP calls: the input gradient's contraction runs over the outputs
VJP = [(300, 3, 60, 200), (300, 3, 150, 200), (40000, 4, 200, 30), (40000, 4, 300, 64), (40000, 4, 300, 80),
       (40000, 40, 300, 128), (40000, 4, 20, 300), (40000, 4, 50, 300), (40000, 40, 100, 300), (40000, 2, 100, 300),
       (40000, 40, 200, 150), (40000, 2, 200, 150),
       *[(3000, 5, k, n) for k in (30, 60, 100) for n in (20, 50, 120)]]


def all_forms():
    out = set()
    for f32 in (True, False):
        for s in FORWARD:
            out |= forward(f32, *s)
        for s in VJP:
            for act in ("silu", "none"):
                out |= vjp(f32, act, *s)
    return out
