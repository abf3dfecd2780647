// Host check of the access test of the checked build (DbgAccess): what counts as
// inside a call's buffers.  Prints "ok <cases>".
#define REPOPS_DEBUG_BOUNDS
#include <cstdio>

#include "internal.cuh"

namespace repops {
int set_cuda_error(cudaError_t) { return REPOPS_ERR_CUDA; }
int status_word_address(unsigned **) { return REPOPS_OK; }
}  // namespace repops

static int cases, bad;

static void expect(bool got, bool want, const char *what) {
    ++cases;
    if (got != want) {
        ++bad;
        std::printf("wrong: %s\n", what);
    }
}

int main() {
    using repops::DbgAccess;
    auto at = [](uintptr_t a) { return reinterpret_cast<void *>(a); };
    DbgAccess d;
    d.reads(at(0x1000), 64);
    d.reads_words(at(0x2003), 6);          // bytes 0x2003 .. 0x2008: words 0x2000 .. 0x200b
    d.writes(at(0x3000), 16);
    d.reads(nullptr, 64);                  // an operand that is not there
    d.writes(at(0x4000), 0);
    d.reads_words(at(0x5001), 0);
    for (uint32_t n : {1u, 2u, 4u, 8u, 16u}) {
        expect(d.may_read(at(0x1000), n), true, "an input's first bytes");
        expect(d.may_read(at(0x1040 - n), n), true, "an input's last bytes");
        expect(d.may_read(at(0x1041 - n), n), false, "one byte behind an input");
        expect(d.may_read(at(0x0fff), n), false, "one byte before an input");
        expect(d.may_write(at(0x1000), n), false, "writing an input");
        expect(d.may_read(at(0x3000), n) && d.may_write(at(0x3000), n), true, "an output");
        expect(d.may_write(at(0x3011 - n), n), false, "one byte behind an output");
        expect(d.may_read(at(0x3011 - n), n), false, "reading one byte behind an output");
        expect(d.may_write(at(0x2fff), n), false, "one byte before an output");
        expect(d.may_read(nullptr, n) || d.may_write(nullptr, n), false, "null");
        expect(d.may_read(at(0x4000), n) || d.may_write(at(0x4000), n), false, "an empty output");
        expect(d.may_read(at(0x5000), n), false, "an empty input");
    }
    for (uintptr_t w : {0x2000u, 0x2004u, 0x2008u}) expect(d.may_read(at(w), 4), true, "a word with a byte of the input");
    for (uintptr_t w : {0x1ffcu, 0x200cu}) expect(d.may_read(at(w), 4), false, "a word without one");
    expect(d.may_read(at(UINTPTR_MAX - 1), 16), false, "the end of memory");
    DbgAccess all;                         // as many buffers as there is room for
    for (int i = 0; i < DbgAccess::kMost; ++i) {
        all.reads(at(0x10000u + 0x100u * i), 16);
        all.writes(at(0x20000u + 0x100u * i), 16);
    }
    for (int i = 0; i < DbgAccess::kMost; ++i) {
        expect(all.may_read(at(0x10000u + 0x100u * i), 16), true, "every input");
        expect(all.may_write(at(0x20000u + 0x100u * i), 16), true, "every output");
    }
    if (bad) return 1;
    std::printf("ok %d\n", cases);
    return 0;
}
