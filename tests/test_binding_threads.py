"""The binding's lookups of torch's functions, made by whichever thread calls
first: at no line may another thread find them half made."""
import sys

import pytest

torch = pytest.importorskip("torch")


def test_first_lookups_are_never_seen_half_made(monkeypatch):
    from prng_seeded_decompress_b200 import build
    build.build()
    from prng_seeded_decompress_b200 import seedlm as sl
    monkeypatch.setattr(sl, "_CODES", {})
    monkeypatch.setattr(sl, "_raw_stream", None)
    monkeypatch.setattr(sl, "_current_device", None)
    seen = []

    def between(frame, event, arg):
        if frame.f_code is sl._bind_torch.__code__:
            # What a call of another thread would use now: _any_dtype() goes by
            # _CODES, _run_on() by _raw_stream.
            seen.append((len(sl._CODES), sl._raw_stream is None or sl._current_device is not None))
        return between

    before = sys.gettrace()
    sys.settrace(between)
    try:
        sl._bind_torch()
    finally:
        sys.settrace(before)
    assert len(seen) > 3 and all(codes in (0, 3) and ready for codes, ready in seen)
    assert sl._raw_stream is not None and sl._current_device is not None
