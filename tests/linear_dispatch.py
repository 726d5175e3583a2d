"""The sizes by which linear attention cuts prompts into parts, restated, so that a
test can say what a batch is cut into and fails when the rule moves away from it."""
import math

SMS = 152


def cut(dt, H, dk, dv):
    """Blocks that the GPU holds, blocks of a part, tokens of a chunk, the least chunks of a part."""
    if dt == "bf16" and min(dk, dv) >= 64:
        return 2 * SMS, H, 64, 2
    return SMS * {128: 4, 64: 6}.get(dk, 8), H * (2 if dv > 64 else 1), 16, 1


def part_chunks(N, B, dt, H, dk, dv):
    """Chunks of a part, 0: segments are whole."""
    blocks, of_part, chunk, least_part = cut(dt, H, dk, dv)
    if B > 1024 or B < 1 or N <= chunk * least_part:
        return 0
    of_64, chunks, share, room = 64 / chunk, N / chunk + 0.5 * B, of_part / blocks, max(1, blocks // of_part)

    def time(parts, of_part):
        waves = parts * share
        return (1.0 if waves <= 1 else waves + 0.5) * of_part
    longest = min(chunks, (1 + 0.55 * math.log2(B)) * chunks / B)
    even = B * share * (chunks / B + 1.5 * of_64)
    least, best, k = max(longest + 1.5 * of_64, even), 0, 2
    while k <= 2 * room + B:
        part = max(int(chunks / k) + 1, least_part)
        rest = chunks / part - 0.5 * B
        if rest > 0:
            t = time(rest + B, part + 1.5 * of_64) + time(rest, 0.5 * part + of_64) + of_64
            if t < least:
                best, least = part, t
        if part == least_part:
            break
        k += k // 16 + 1
    if not best and B > 1 and even >= 12 * of_64:
        best = int(1.2 * max(longest, even) + 4 * of_64)
    return best if best * chunk < N else 0


def workspace(N, B, dt, H, dk, dv):
    """Bytes that this batch needs: a decay and a state for each part and head."""
    part = part_chunks(N, B, dt, H, dk, dv)
    parts = N // (cut(dt, H, dk, dv)[2] * part) + 2 * B if part else 0
    return (parts * H * 8 + 255) // 256 * 256 + parts * H * dk * dv * 4 if parts else 0
