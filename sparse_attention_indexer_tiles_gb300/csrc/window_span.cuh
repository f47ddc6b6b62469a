// The tokens of a request in a call of the windowed attention (attention_window*.cu).
#pragma once

#include "common.cuh"
#include "window.cuh"

namespace idx {

struct Span {
    int first, count;  // tokens
    int len;           // cached slots, the new tokens' among them
};
IDX_DEVI Span span_of(const WindowArgs& a, int b, bool report) {
    Span s;
    int end;
    if (a.q_start) {
        s.first = a.q_start[b];
        end = a.q_start[b + 1];
    } else {
        const int per = a.T / a.B;
        s.first = b * per;
        end = s.first + per;
    }
    s.len = a.lens[b];
    const bool wrong = s.first < 0 || end < s.first || end > a.T;
    if (report && (wrong || end - s.first > a.max_q || s.len < 0 || s.len > a.max_len))
        raise_status(a.d_status, IDX_DEV_RANGE);
    s.count = wrong ? 0 : min(end - s.first, a.max_q);
    if (wrong) s.first = 0;
    s.len = min(max(s.len, 0), a.max_len);
    return s;
}

}  // namespace idx
