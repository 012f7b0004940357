// The verification kernels as a CPU library: one call runs them in a process of its
// own, every array's end (every row's, of the logits) at a page that may not be
// touched, and the rows of `drafted` that are marked likewise altogether.
#include "q4_0_verify.hip"

#include <sys/mman.h>
#include <sys/wait.h>
#include <unistd.h>

namespace q4 {
static int g_cus;
DeviceShape device_shape() { return {g_cus, 1}; }
}  // namespace q4

namespace {

constexpr size_t kPage = 4096;

// `bytes` bytes that end where a page without access begins.
uint8_t *guarded(const void *from, size_t bytes) {
    const size_t room = (bytes + kPage - 1) / kPage * kPage;
    uint8_t *p = (uint8_t *)mmap(nullptr, room + kPage, PROT_READ | PROT_WRITE,
                                 MAP_PRIVATE | MAP_ANONYMOUS, -1, 0);
    if (p == MAP_FAILED || mprotect(p + room, kPage, PROT_NONE)) _exit(4);
    p += room - bytes;
    if (from)
        memcpy(p, from, bytes);
    else
        memset(p, 0xFF, bytes);
    return p;
}

// n rows of `bytes` bytes, each up to such a page; those marked have none.
uint8_t *guarded_rows(const uint8_t *from, size_t n, size_t bytes, size_t pitch,
                      const uint8_t *marked) {
    uint8_t *p = (uint8_t *)mmap(nullptr, n * pitch, PROT_READ | PROT_WRITE,
                                 MAP_PRIVATE | MAP_ANONYMOUS, -1, 0);
    if (p == MAP_FAILED) _exit(4);
    for (size_t t = 0; t < n; ++t) {
        uint8_t *row = p + t * pitch;
        memcpy(row + pitch - kPage - bytes, from + t * bytes, bytes);
        const bool none = marked && marked[t];
        if (mprotect(none ? row : row + pitch - kPage, none ? pitch : kPage, PROT_NONE)) _exit(4);
    }
    return p + pitch - kPage - bytes;
}

}  // namespace

// The status of the process (0: done), as waitpid gives it.  logits and drafted: dense rows.
extern "C" int host_verify(const void *logits, const void *drafted, const uint8_t *marked, int f16,
                           int64_t vocab, const int32_t *tokens, const int32_t *q_start, int64_t n,
                           int64_t batch, const float *heat, const float *uniform, int cus,
                           int32_t *out) {
    int32_t *shared = (int32_t *)mmap(nullptr, 8 * batch, PROT_READ | PROT_WRITE,
                                      MAP_SHARED | MAP_ANONYMOUS, -1, 0);
    if (shared == MAP_FAILED) return -1;
    const pid_t child = fork();
    if (child < 0) return -1;
    if (child == 0) {
        q4::g_cus = cus;
        const size_t row = (size_t)vocab * (f16 ? 2 : 4);
        const size_t pitch = (row + kPage - 1) / kPage * kPage + kPage;
        q4::VerifyArgs a = {};
        a.logits = guarded_rows((const uint8_t *)logits, n, row, pitch, nullptr);
        if (drafted) a.drafted = guarded_rows((const uint8_t *)drafted, n, row, pitch, marked);
        a.stride = a.drafted_stride = (int64_t)(pitch / (f16 ? 2 : 4));
        a.vocab = (int)vocab, a.n = (int)n, a.batch = (int)batch;
        a.tokens = (const int32_t *)guarded(tokens, 4 * n);
        a.q_start = (const int32_t *)guarded(q_start, 4 * (batch + 1));
        a.heat = heat ? (const float *)guarded(heat, 4 * batch) : nullptr;
        a.uniform = (const float *)guarded(uniform, 8 * n);
        a.accepted = (int32_t *)guarded(nullptr, 4 * batch);
        a.next = (int32_t *)guarded(nullptr, 4 * batch);
        // (whole multiples of 8 bytes: the kernels' own alignment is kept)
        void *ws = guarded(nullptr, q4::verify_workspace_bytes(n, batch, vocab, drafted != nullptr));
        if (q4::launch_verify(a, f16, ws, nullptr) != hipSuccess) _exit(3);
        memcpy(shared, a.accepted, 4 * batch);
        memcpy(shared + batch, a.next, 4 * batch);
        _exit(0);
    }
    int status = -1;
    if (waitpid(child, &status, 0) != child) status = -1;
    memcpy(out, shared, 8 * batch);
    munmap(shared, 8 * batch);
    return status;
}
