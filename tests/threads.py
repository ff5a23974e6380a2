"""Functions run in threads of their own, at once: what they return, and what they raise
as the caller's error."""

from __future__ import annotations

import threading


def together(*works):
    results, errors = [None] * len(works), []
    start = threading.Barrier(len(works))

    def run(i):
        try:
            start.wait()
            results[i] = works[i]()
        except BaseException as e:  # noqa: BLE001
            errors.append((i, e))

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(works))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if errors:
        i, e = errors[0]
        raise AssertionError(f"thread {i} raised {type(e).__name__}: {e} ({len(errors)} of {len(works)} threads)") from e
    return results
