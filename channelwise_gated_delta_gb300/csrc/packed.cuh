// packed.cuh -- sequences of rows for the operators around the recurrence:
// dense batches (N sequences of T rows) or packed ones (offsets on the host),
// cut into units of a fixed number of rows that the CTAs of a launch take.
//
// A launch gets the offsets by value, as part of its arguments: no copy from
// host memory and no workspace, so a packed call can be captured into a graph
// and two captured calls share nothing.  A batch of more than kTableSeqs
// sequences is several launches.
#pragma once

#include <stdint.h>

#include "gdr.h"
#include "host_checks.h"

namespace gdr {

constexpr int kTableSeqs = 256;

struct SeqTable {
    int n;         // sequences of this launch
    int seq0;      // the first one's index in the batch
    int unit0;     // the first unit's index in the batch
    int T;         // rows of every sequence (dense), -1: by the tables
    int units_of;  // units of every sequence (dense)
    int cu[kTableSeqs + 1];    // first row of each
    int unit[kTableSeqs + 1];  // first unit of each
};

struct SeqUnit {
    int seq;         // index in the batch
    int unit;        // unit of the sequence
    int len;         // rows of the sequence
    long long row0;  // its first row
};

__device__ __forceinline__ SeqUnit find_unit(const SeqTable &t, int u) {
    SeqUnit r;
    if (t.T >= 0) {
        const int s = u / t.units_of;
        r.seq = t.seq0 + s;
        r.unit = u - s * t.units_of;
        r.len = t.T;
        r.row0 = (long long)r.seq * t.T;
        return r;
    }
    int lo = 0, hi = t.n - 1;  // the last sequence whose first unit is not behind u
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.unit[mid] <= u)
            lo = mid;
        else
            hi = mid - 1;
    }
    r.seq = t.seq0 + lo;
    r.unit = u - t.unit[lo];
    r.row0 = t.cu[lo];
    r.len = t.cu[lo + 1] - t.cu[lo];
    return r;
}

// ---- host side
// Offsets of a packed batch: start at 0, never fall.
inline gdr_status check_offsets(const int *cu, int N) {
    if (cu[0] != 0) return GDR_ERR_SHAPE;
    for (int n = 0; n < N; ++n)
        if (cu[n + 1] < cu[n]) return GDR_ERR_SHAPE;
    return GDR_OK;
}
// Units of a sequence; one without rows still has one (its state is copied).
inline long long units_of_rows(long long rows, int unit_rows) {
    return rows <= unit_rows ? 1 : (rows + unit_rows - 1) / unit_rows;
}
inline long long count_units(const int *cu, int N, int T, int unit_rows) {
    if (!cu) return N * units_of_rows(T, unit_rows);
    long long u = 0;
    for (int n = 0; n < N; ++n) u += units_of_rows(cu[n + 1] - cu[n], unit_rows);
    return u;
}
// Calls launch(table, units) for the batch's launches; stops at an error.
template <typename F>
cudaError_t for_sequences(const int *cu, int N, int T, int unit_rows, F launch) {
    SeqTable t;
    if (!cu) {
        t.n = N;
        t.seq0 = 0;
        t.unit0 = 0;
        t.T = T;
        t.units_of = (int)units_of_rows(T, unit_rows);
        return launch(t, (long long)N * t.units_of);
    }
    long long before = 0;
    for (int n0 = 0; n0 < N; n0 += kTableSeqs) {
        t.n = N - n0 < kTableSeqs ? N - n0 : kTableSeqs;
        t.seq0 = n0;
        t.T = -1;
        t.units_of = 0;
        long long u = 0;
        for (int i = 0; i < t.n; ++i) {
            t.cu[i] = cu[n0 + i];
            t.unit[i] = (int)u;
            u += units_of_rows(cu[n0 + i + 1] - cu[n0 + i], unit_rows);
        }
        t.cu[t.n] = cu[n0 + t.n];
        t.unit[t.n] = (int)u;
        t.unit0 = (int)before;
        before += u;
        const cudaError_t e = launch(t, u);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

// Whether n rows `ld` elements apart can be addressed at all.
inline bool rows_fit(long long n, long long ld) {
    return n <= 0 || ld <= (1LL << 58) / n;
}
// Rows of `width` bytes, `ld` bytes apart.
struct RowSet {
    const void *p;
    size_t width, ld;
    long long n;
};
inline RowSet packed_rows(const void *p, size_t bytes) { return RowSet{p, bytes, bytes, p ? 1 : 0}; }
// Whether two sets of rows share memory.  Rows at the same distance may lie
// between each other's (parts of one wider tensor).
inline bool rows_overlap(const RowSet &a, const RowSet &b) {
    if (!a.p || !b.p || a.n <= 0 || b.n <= 0 || !a.width || !b.width) return false;
    const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
    const uintptr_t a1 = a0 + (a.n - 1) * a.ld + a.width, b1 = b0 + (b.n - 1) * b.ld + b.width;
    if (a1 <= b0 || b1 <= a0) return false;
    if (a.ld != b.ld || a.n == 1 || b.n == 1) return true;
    const size_t off = b0 >= a0 ? (b0 - a0) % a.ld : (a.ld - (a0 - b0) % a.ld) % a.ld;
    return off < a.width || off + b.width > a.ld;
}

}  // namespace gdr
