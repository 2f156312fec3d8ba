"""The first calls of two threads at once: whoever finds the library loaded
finds the packed calls' tables too."""
import threading

import causal_depthwise_short_conv1d_amd as S


def test_packed_calls_are_there_when_the_library_is(monkeypatch):
    found = []

    def other_thread():
        S.load_library()
        found.extend(fn in S._packed for fn in ("gdr_fwd_varlen", "gdr_update"))

    class Table(dict):
        first = True

        def update(self, *a):
            if self.first:                             # a second thread's first call comes in here
                self.first = False
                t = threading.Thread(target=other_thread)
                t.start()
                t.join()
            super().update(*a)

    monkeypatch.setattr(S, "_lib", None)
    monkeypatch.setattr(S, "_packed", Table())
    S.load_library()
    assert found == [True, True]
