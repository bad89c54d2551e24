// Scratch buffers that grow: an address and the elements that it holds, which only ever change together.
#pragma once
#include <stddef.h>

namespace adp {

template <class T>
struct Grown {
  T* p = nullptr;
  size_t n = 0;
  operator T*() const { return p; }
};

// Room for n elements at least.  release(p) frees the old buffer, allocate(&p, n) makes the new one; both return a status,
// 0 for success, which is passed on.  Where they fail, the buffer is what it was or empty.
template <class T, class Allocate, class Release>
int grow(Grown<T>* b, size_t n, Allocate allocate, Release release) {
  if (n <= b->n) return 0;
  if (b->p) {
    const int rc = release(b->p);
    if (rc) return rc;
    *b = Grown<T>();
  }
  T* p = nullptr;
  const int rc = allocate(&p, n);
  if (!rc) b->p = p, b->n = n;
  return rc;
}

}  // namespace adp
