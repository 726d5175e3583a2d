"""The sizes by which the state space calls choose a variant, restated, so that
a test can say which one it reaches and fails when a rule moves away from it."""
SMS = 152
INT_MAX = 2 ** 31 - 1


def _up(a, b):
    return -(-a // b)


# ---------------------------------------------------------------- convolution
def conv_tile(dt, N, D):
    """Tokens of a tile of a prompt (channels by fours)."""
    want = SMS * (7 if dt == "bf16" else 5) * 128
    return min(max(N * _up(D, 4) // want // 8 * 8 + 8, 8), 48)


# ---------------------------------------------------------------- scan, steps
def step_rows(dt, S, B, D, G=1, table=True):
    """The most rows that a block takes; table: rows of any number of tokens."""
    chans = 256 // (S // 8)
    gx = G * _up(D // G, chans) if table else _up(D, chans)
    room = SMS * (4 if table or dt == "bf16" else 3)
    least, best, groups = _up(B, 128), None, 0
    for w in range(1, 5):
        gy = min(max(w * room // gx, least), max(B, least))
        cost = _up(gx * gy, room) * (_up(B, gy) + 2)
        if best is None or cost < best:
            best, groups = cost, gy
    return _up(B, groups)


# -------------------------------------------------------------- scan, prompts
def scan_blocks(D, S, G=1):
    """Blocks across the channels."""
    return G * _up(D // G, 256 // (S // 8))


def scan_part(N, B, D, S, G=1):
    """Tokens of a part, 0: segments are walked whole."""
    nblk, room = scan_blocks(D, S, G), SMS * (5 if S <= 32 else 4)
    if 2 * B * nblk > INT_MAX:
        return 0
    part = _up(N * nblk, 2 * room)
    if B * nblk >= 3 * SMS:
        part = max(part, _up(2 * N, B))
    part = _up(part, 16) * 16
    while part < 32 or part * part < N:
        part += 16
    if part >= N:
        return 0
    while (N // part + 2 * B) * nblk > INT_MAX:
        part *= 2
    return part


def scan_joined(N, B, D, S, G=1):
    """Whether a launch of its own joins the parts' states."""
    part = scan_part(N, B, D, S, G)
    return bool(part) and N // part > 16 * B


def scan_listed(N, B, D, S, G=1):
    """Whether the parts are listed first, the long ones in front."""
    return bool(scan_part(N, B, D, S, G)) and B > 1 and N * scan_blocks(D, S, G) >= 100000
