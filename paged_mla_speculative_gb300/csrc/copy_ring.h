// Copies through two buffers in turn, one filled while the other is written
// out.  Plain C++, so that what it does when a copy is late runs on the host
// too (there is no late copy to be had on a GPU).
#pragma once

#ifdef __CUDACC__
#define MLAV_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define MLAV_HOST_DEVICE inline
#endif

namespace mlav {

// Pieces 0 .. total - 1 (at least one), piece i in buffer i % 2.  Ops: load(i)
// starts the copy in, landed(i) asks for its end, store(i) starts the copy
// out, drain() returns when every copy out has read its buffer, now() is a
// clock, late() reports a copy in that took longer than `limit`.
// A late piece has as long again and is then used like any other.  One that
// has not landed by then ends the run, and so that nothing lands in a buffer
// that is given up, the piece loaded behind it gets its time first.
template <class Ops>
MLAV_HOST_DEVICE void copy_through_two(Ops& ops, int total, long long limit) {
  ops.load(0);
  for (int i = 0; i < total; ++i) {
    if (i + 1 < total) {
      // The other buffer is free once its last piece has been read out.
      if (i) ops.drain();
      ops.load(i + 1);
    }
    const long long t0 = ops.now();
    bool late = false;
    while (!ops.landed(i)) {
      const long long t = ops.now() - t0;
      if (t > limit && !late) {
        ops.late();
        late = true;
      }
      if (t > 2 * limit) {
        const long long t1 = ops.now();
        while (i + 1 < total && !ops.landed(i + 1) && ops.now() - t1 <= limit) {
        }
        return;
      }
    }
    ops.store(i);
  }
}

}  // namespace mlav
