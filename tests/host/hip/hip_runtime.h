// A workgroup's threads on the CPU, for kernels compiled as plain C++: every lane is
// a context of its own, a wave of 64 lanes meets at each operation that moves
// values between lanes, a workgroup at its barriers.  Workgroups run one after
// another.  Lanes that have returned take part in nothing.  Only what the kernels
// that are tested this way use is here.
#pragma once

#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>
#include <ucontext.h>

#include <functional>
#include <vector>

#define __global__
#define __device__
#define __host__
#define __forceinline__ inline
#define __shared__ static
#define __launch_bounds__(...)

struct dim3 {
    uint32_t x, y, z;
    dim3(uint32_t a = 1, uint32_t b = 1, uint32_t c = 1) : x(a), y(b), z(c) {}
};
typedef int hipError_t;
typedef void *hipStream_t;
constexpr hipError_t hipSuccess = 0;
inline hipError_t hipGetLastError() { return hipSuccess; }

namespace host {

constexpr int kWave = 64;

struct Lane {
    ucontext_t at;
    std::vector<char> stack;
    int x;
    bool done;
    uint64_t wave_turn, group_turn;  // meetings this lane has been to
};
// Where some lanes meet: all that have not returned.
struct Meeting {
    int here = 0, live = 0;
    uint64_t turn = 0;
    uint64_t said[kWave], heard[2][kWave], mask[2], saying = 0;
    void close() {
        if (live == 0 || here < live) return;
        memcpy(heard[turn & 1], said, sizeof(said));
        mask[turn & 1] = saying;
        saying = 0;
        here = 0;
        ++turn;
    }
};
struct State {
    dim3 grid, group, block;
    std::vector<Lane> lanes;
    std::vector<Meeting> waves;
    Meeting all;
    ucontext_t back;
    Lane *me = nullptr;
    std::function<void()> body;
};
inline State g;

inline void wait() { swapcontext(&g.me->at, &g.back); }

// What every live lane of the wave says.
struct Heard {
    const uint64_t *of;
    uint64_t mask;
    bool has(int lane) const { return mask >> lane & 1; }
};
inline Heard meet(uint64_t value) {
    Lane *me = g.me;
    Meeting &w = g.waves[me->x / kWave];
    const int lane = me->x % kWave;
    const uint64_t turn = me->wave_turn++;
    w.said[lane] = value;
    w.saying |= uint64_t(1) << lane;
    ++w.here;
    w.close();
    while (w.turn == turn) wait();
    return {w.heard[turn & 1], w.mask[turn & 1]};
}
inline void barrier() {
    const uint64_t turn = g.me->group_turn++;
    ++g.all.here;
    g.all.close();
    while (g.all.turn == turn) wait();
}

inline void lane_main() {
    g.body();
    Lane *me = g.me;
    me->done = true;
    for (Meeting *m : {&g.waves[me->x / kWave], &g.all}) {
        --m->live;
        m->close();
    }
    for (;;) wait();
}

inline void run_workgroup() {
    const int count = (int)g.group.x;
    g.waves.assign((count + kWave - 1) / kWave, Meeting());
    g.all = Meeting();
    g.lanes.resize(count);
    for (int i = 0; i < count; ++i) {
        Lane &l = g.lanes[i];
        if (l.stack.empty()) l.stack.resize(128 * 1024);
        l.x = i;
        l.done = false;
        l.wave_turn = l.group_turn = 0;
        ++g.waves[i / kWave].live;
        ++g.all.live;
        getcontext(&l.at);
        l.at.uc_stack.ss_sp = l.stack.data();
        l.at.uc_stack.ss_size = l.stack.size();
        l.at.uc_link = nullptr;
        makecontext(&l.at, lane_main, 0);
    }
    for (int left = count, idle = 0; left > 0;) {
        left = 0;
        for (Lane &l : g.lanes) {
            if (l.done) continue;
            g.me = &l;
            swapcontext(&g.back, &l.at);
            left += !l.done;
        }
        if (++idle > 100000000) abort();
    }
}

template <typename F> void launch(dim3 grid, dim3 group, F body) {
    g.grid = grid;
    g.group = group;
    g.body = body;
    for (uint32_t z = 0; z < grid.z; ++z)
        for (uint32_t y = 0; y < grid.y; ++y)
            for (uint32_t x = 0; x < grid.x; ++x) {
                g.block = dim3(x, y, z);
                run_workgroup();
            }
}

// Moves within rows of 16 lanes, and a row's (two rows') last lane to the next.
inline int moved_from(int lane, int ctrl) {
    const int row = lane / 16, in = lane % 16;
    if (ctrl == 0xE4) return lane;
    if (ctrl > 0x110 && ctrl < 0x120) return in >= ctrl - 0x110 ? lane - (ctrl - 0x110) : -1;
    if (ctrl > 0x120 && ctrl < 0x130) return row * 16 + (in - (ctrl - 0x120) + 16) % 16;
    if (ctrl == 0x142) return row ? row * 16 - 1 : -1;
    if (ctrl == 0x143) return row >= 2 ? 31 : -1;
    abort();
}
inline int dpp(int old, int src, int ctrl, int rows, bool zero) {
    const Heard h = meet((uint32_t)src);
    const int lane = g.me->x % kWave, from = moved_from(lane, ctrl);
    if (!(rows >> lane / 16 & 1)) return old;
    if (from < 0 || !h.has(from)) return zero ? 0 : old;
    return (int)(uint32_t)h.of[from];
}
struct Pair {
    uint32_t v[2];
    uint32_t operator[](int i) const { return v[i]; }
};
inline Pair swapped(uint32_t a, uint32_t b, int rows) {
    const Heard h = meet((uint64_t)a << 32 | b);
    const int lane = g.me->x % kWave;
    const int odd = lane / rows & 1;
    const uint32_t first = odd ? (uint32_t)h.of[lane - rows] : a;
    const uint32_t second = odd ? b : (uint32_t)(h.of[lane + rows] >> 32);
    return {{first, second}};
}

inline int first(int x) {
    const Heard h = meet((uint32_t)x);
    return (int)(uint32_t)h.of[__builtin_ctzll(h.mask)];
}

}  // namespace host

#define threadIdx (dim3((uint32_t)host::g.me->x, 0, 0))
#define blockIdx (host::g.block)
#define blockDim (host::g.group)
#define gridDim (host::g.grid)
#define hipLaunchKernelGGL(kernel, grid, group, lds, stream, ...) \
    host::launch(grid, group, [=] { kernel(__VA_ARGS__); })

template <typename T> inline T min(T a, T b) { return b < a ? b : a; }
template <typename T> inline T max(T a, T b) { return a < b ? b : a; }
inline void __syncthreads() { host::barrier(); }
inline uint64_t __ballot(bool x) {
    const host::Heard h = host::meet(x);
    uint64_t r = 0;
    for (int i = 0; i < 64; ++i)
        if (h.has(i) && h.of[i]) r |= uint64_t(1) << i;
    return r;
}
inline bool __all(bool x) {
    const host::Heard h = host::meet(x);
    for (int i = 0; i < 64; ++i)
        if (h.has(i) && !h.of[i]) return false;
    return true;
}
inline int __shfl_xor(int x, int m) {
    const host::Heard h = host::meet((uint32_t)x);
    return (int)(uint32_t)h.of[(host::g.me->x % 64) ^ m];
}
inline int __popcll(uint64_t x) { return __builtin_popcountll(x); }
inline int __ffsll(unsigned long long x) { return __builtin_ffsll((long long)x); }
inline int __clzll(uint64_t x) { return x ? __builtin_clzll(x) : 64; }
inline int atomicMax(int *p, int x) {
    const int was = *p;
    if (x > was) *p = x;
    return was;
}
#define __builtin_amdgcn_sched_barrier(x)
#define __builtin_amdgcn_perm(a, b, c) (abort(), 0u)
#define __builtin_amdgcn_mov_dpp(src, ctrl, rows, banks, zero) host::dpp(0, src, ctrl, rows, true)
#define __builtin_amdgcn_update_dpp(old, src, ctrl, rows, banks, zero) \
    host::dpp(old, src, ctrl, rows, zero)
#define __builtin_amdgcn_readlane(x, lane) ((int)(uint32_t)host::meet((uint32_t)(x)).of[lane])
#define __builtin_amdgcn_readfirstlane(x) host::first(x)
#define __builtin_amdgcn_permlane16_swap(a, b, c, d) host::swapped(a, b, 16)
#define __builtin_amdgcn_permlane32_swap(a, b, c, d) host::swapped(a, b, 32)
