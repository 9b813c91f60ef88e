// What the operators' entry points share: checks of their buffers, and the parts of
// a context they use.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <initializer_list>
#include <string>

struct moe_ctx;

namespace moe {

// Whether all addresses are multiples of an element's size (null is).
inline bool whole(std::initializer_list<const void *> ptrs, uintptr_t size) {
    for (const void *p : ptrs)
        if ((uintptr_t)p & (size - 1)) return false;
    return true;
}

// Bytes that an operator reads or writes (none without an address).
struct Span {
    const void *p;
    size_t n;
    bool meets(const Span &o) const {
        const uintptr_t a = (uintptr_t)p, b = (uintptr_t)o.p;
        return p && o.p && a < b + o.n && b < a + n;
    }
};

// Whether no output meets an input or another output.  Rows are worked on by
// independent warps and CTAs: what one writes over bytes that another has yet to
// read is a race.
inline bool apart(std::initializer_list<Span> in, std::initializer_list<Span> out) {
    for (const Span *o = out.begin(); o != out.end(); ++o) {
        for (const Span &i : in)
            if (o->meets(i)) return false;
        for (const Span *q = out.begin(); q != o; ++q)
            if (o->meets(*q)) return false;
    }
    return true;
}

// What an operator uses of a context.
struct OpContext {
    cudaStream_t stream;
    int device, n_sm;
    int *error;  // device error word, reported by the next cache_step or miss_drain
};
OpContext op_context(const moe_ctx *ctx);
// Keeps the message (without a context: the host thread's) and returns the code.
int op_fail(moe_ctx *ctx, int code, const std::string &msg);

}  // namespace moe
